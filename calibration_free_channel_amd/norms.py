"""The norms before and after a block.

The work runs in the library's HIP kernels (cfr_block_norm_in and
cfr_block_norm_out, include/cfr.h); arguments are checked in csrc/py_ops.cpp.
"""
from __future__ import annotations

from ._ext import on_stream, ops

GATE_ACTS = {"none": 0, "sigmoid": 1, "silu": 2, "tanh": 3}


def block_norm_in(x, weight=None, eps=1e-6, offset=0.0, out=None, dtype=None, stream=None):
    """u = x / sqrt(mean(x^2) + eps) * (offset + weight) over the last
    dimension of x [..., cols] (float32, bfloat16 or float16), in `dtype`
    (x's by default) or in `out`'s; `out` may be x.  Without a weight the
    factor is one.  Sums in float32.  Inference only: tensors that need a
    gradient are refused while gradients are recorded."""
    if stream is not None:
        return on_stream(stream, x, ops.norm_in, x, weight, eps, offset, out, dtype)
    return ops.norm_in(x, weight, eps, offset, out, dtype)


def block_norm_out(y, x, post_weight=None, post_norm=True, gate=None, gate_act="none", out_scale=1.0,
                   resid_scale=1.0, next_weight=None, next_norm=False, eps=1e-6, offset=0.0, out=None, next_out=None,
                   next_dtype=None, stream=None):
    """The residual stream after a block, and the next block's input:

        v = y / sqrt(mean(y^2) + eps) * (offset + post_weight)   (y itself without post_norm)
        s = resid_scale * x + out_scale * act(gate) * v
        u = s / sqrt(mean(s^2) + eps) * (offset + next_weight)   (with next_norm)

    y [..., cols] is the block's output, x of the same shape (and any of the
    three types) the residual stream.  gate, of y's type: [cols] (or [1, cols])
    for a gate per channel, [..., 1] with y's leading sizes for one per token,
    y's shape for one per value; gate_act is "none", "sigmoid", "silu" or
    "tanh".  Returns s in x's type (in `out`, which may be x), and with
    next_norm the pair (s, u), u in next_dtype (y's by default) or in
    `next_out`.  Inference only, as block_norm_in."""
    act = GATE_ACTS.get(gate_act)
    if act is None:
        raise ValueError(f"gate_act must be one of {sorted(GATE_ACTS)}")
    if stream is not None:
        return on_stream(stream, y, ops.norm_out, y, x, post_weight, post_norm, gate, act, out_scale, resid_scale,
                         next_weight, next_norm, eps, offset, out, next_out, next_dtype)
    return ops.norm_out(y, x, post_weight, post_norm, gate, act, out_scale, resid_scale, next_weight, next_norm, eps,
                        offset, out, next_out, next_dtype)
