"""The routed experts on microscaled 4-bit weights, for any number of tokens.

The work runs in the library's HIP kernels (cfr_build_experts and
cfr_experts_forward, include/cfr.h); forward's arguments are checked in
csrc/py_ops.cpp.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from ._ext import on_stream, ops
from ._lib import CfrExpertsConfig, check, load


@dataclass(frozen=True)
class ExpertsConfig:
    hidden: int
    n_experts: int
    inter: int
    top: int
    max_tokens: int = 64
    device: int = 0

    def c(self) -> CfrExpertsConfig:
        return CfrExpertsConfig(self.hidden, self.n_experts, self.inter, self.top, self.max_tokens, self.device)


def _weights(pair, lead, cols, name, device):
    codes, scales = pair
    ptrs = []
    for t, n, what in ((codes, (cols + 1) // 2, "codes"), (scales, (cols + 31) // 32, "scales")):
        shape = (*lead, n)
        if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or not t.is_cuda or t.device.index != device:
            raise ValueError(f"{name} {what}: expected a uint8 tensor on device {device}")
        if tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} {what}: expected a contiguous tensor of shape {shape}, got {tuple(t.shape)}")
        ptrs.append(t.data_ptr())
    return ptrs


class Experts:
    """One layer's routed experts on MXFP4 weights.  Owns device memory until
    close(): the weights, and a workspace for max_tokens tokens (about 6 hidden
    + top (6 inter + 4 hidden) bytes each).  Calls on one object share the
    workspace: order them on one stream."""

    def __init__(self, handle: ctypes.c_void_p, cfg: ExpertsConfig):
        self._h = handle
        self.cfg = cfg

    @classmethod
    def build(cls, cfg: ExpertsConfig, gate, up, down, stream=None) -> "Experts":
        """gate, up and down are (codes, scales) pairs as mx4_quantize gives
        them, of [E, I, H], [E, I, H] and [E, H, I] weights.  They are copied
        into the layout of the products and may be freed afterwards."""
        if stream is not None and stream.device != torch.device("cuda", cfg.device):
            raise ValueError(f"stream: on device {stream.device}, not the tensors' own")
        E, I, H = cfg.n_experts, cfg.inter, cfg.hidden
        ptrs = [*_weights(gate, (E, I), H, "gate", cfg.device), *_weights(up, (E, I), H, "up", cfg.device),
                *_weights(down, (E, H), I, "down", cfg.device)]
        st = (stream or torch.cuda.current_stream(cfg.device)).cuda_stream
        h = ctypes.c_void_p()
        check(load().cfr_build_experts(ctypes.byref(cfg.c()), *ptrs, st, ctypes.byref(h)))
        return cls(h, cfg)

    def close(self):
        if self._h is not None and self._h.value:
            load().cfr_experts_free(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, x, expert_ids, gate_w, out=None, stream=None):
        """y [tokens, hidden] of x [tokens, hidden] (float32, bfloat16 or
        float16; rows may be strided): the sum over a token's slots of gate_w
        times the slot's expert's down(silu(gate(x)) * up(x)), in x's type.
        expert_ids int32 [tokens, top] (negative: an empty slot), gate_w
        float32 [tokens, top].  Inference only: tensors that need a gradient
        are refused while gradients are recorded.

        x's type chooses what is kept between the products: silu(gate(x)) *
        up(x) has 24 bits for float32, 16 for float16, and for bfloat16 8 in
        calls of more than 64 slots (16 below), where a slot's values also
        have 11 before they are summed in float32."""
        c = self.cfg
        args = (self._h.value if self._h else None, c.hidden, c.top, c.device, x, expert_ids, gate_w, out)
        if stream is not None:
            return on_stream(stream, x, ops.experts_forward, *args)
        return ops.experts_forward(*args)

    def status(self) -> int:
        """Bit 0: an expert id of n_experts or more was skipped since the last
        status().  Waits for the device."""
        f = ctypes.c_int32()
        check(load().cfr_experts_status(self._h, ctypes.byref(f)))
        return f.value
