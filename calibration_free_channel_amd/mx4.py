"""Microscaled 4-bit floats (MXFP4): rows of values to codes and scales, and back.

The work runs in the library's HIP kernels (cfr_mx4_quantize and
cfr_mx4_dequantize, include/cfr.h); arguments are checked in csrc/py_ops.cpp.
"""
from __future__ import annotations

import torch

from ._ext import on_stream, ops


def mx4_quantize(x, out=None, stream=None):
    """Codes uint8 [..., ceil(cols/2)] and scales uint8 [..., ceil(cols/32)] of
    x [..., cols] (float32, bfloat16 or float16): per 32 values of a row the
    scale 2^(floor(log2 max|x|) - 2) as a byte with bias 127, and each value
    over it as the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with its sign (ties to
    the even code).  `out`: a (codes, scales) tuple to write.  No gradient
    passes through the codes."""
    if stream is not None:
        return on_stream(stream, x, ops.quantize, x, out)
    return ops.quantize(x, out)


def mx4_dequantize(codes, scales, cols, dtype=torch.float32, out=None, stream=None):
    """The values [..., cols] that codes and scales (of mx4_quantize) stand
    for, in `dtype` or in `out`'s; NaN where a scale byte is 255.  Inference
    only: an `out` that needs a gradient is refused while gradients are
    recorded."""
    if stream is not None:
        return on_stream(stream, codes, ops.dequantize, codes, scales, cols, dtype, out)
    return ops.dequantize(codes, scales, cols, dtype, out)
