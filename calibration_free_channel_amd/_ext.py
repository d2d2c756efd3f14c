"""The extension module _ops.so and what its calls share."""
from __future__ import annotations

import os

import torch

from . import _lib


def _current_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


if not os.path.exists(os.path.join(_lib.HERE, "_ops.so")):
    raise RuntimeError("_ops.so is missing: build it with `python -m calibration_free_channel_amd.build`")
_lib.load()
from . import _ops as ops  # noqa: E402


def _check_torch(built, running):
    # the module reads tensors as that torch's headers lay them out
    if built != running:
        raise RuntimeError(f"_ops.so was built for torch {built}, this is {running}: "
                           "build it again with `python -m calibration_free_channel_amd.build`")


_check_torch(ops.torch, str(torch.__version__))

# torch's own way to the current stream's handle builds no Stream object, 1 us less per call
ops.init(getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream), _lib.check)


def on_stream(stream, like, call, *args):
    """call(*args) with its launches and outputs on the caller's stream, and
    the allocator told that this stream uses the tensors."""
    if not isinstance(like, torch.Tensor) or not like.is_cuda or stream.device != like.device:
        raise ValueError(f"stream: on device {stream.device}, not the tensors' own")
    with torch.cuda.stream(stream):
        result = call(*args)
    for t in (*args, result):
        for s in t if isinstance(t, tuple) else (t,):
            if isinstance(s, torch.Tensor) and s.is_cuda:
                s.record_stream(stream)
    return result
