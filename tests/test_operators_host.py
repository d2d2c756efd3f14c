"""Refusals of the operators around the block, checked without a GPU: every
argument error is found on the host before anything is launched."""
import ctypes

import pytest

from calibration_free_channel_amd._lib import CFR_BF16, CFR_F32, CfrError, CfrExpertsConfig, CfrNormOutArgs, check, load

P = ctypes.c_void_p(4096)  # never dereferenced: the calls below fail before a launch


def _refused(rc, code=-1):
    with pytest.raises(CfrError) as ei:
        check(rc)
    assert ei.value.code == code and str(ei.value)


@pytest.mark.parametrize("args", [(P, 9, 4, 32, 32), (P, CFR_F32, -1, 32, 32), (P, CFR_F32, 4, -32, 32)])
def test_mx4_refusals(args):
    _refused(load().cfr_mx4_quantize(*args, P, P, 0, None))
    x, dt, rows, cols, stride = args
    _refused(load().cfr_mx4_dequantize(P, P, rows, cols, x, dt, stride, 0, None))


def test_mx4_sizes_pointers_and_strides():
    q = load().cfr_mx4_quantize
    _refused(q(P, CFR_F32, (1 << 31) - 1, 64, 64, P, P, 0, None), -4)  # 2^32 blocks
    _refused(q(P, CFR_F32, 1 << 40, 32, 32, P, P, 0, None), -4)
    _refused(q(P, CFR_F32, 1, 1 << 40, 1 << 40, P, P, 0, None), -4)
    _refused(q(None, CFR_F32, 4, 64, 64, P, P, 0, None))
    _refused(q(P, CFR_F32, 4, 64, 64, None, P, 0, None))
    _refused(q(P, CFR_F32, 4, 64, 64, P, None, 0, None))
    _refused(q(P, CFR_F32, 4, 64, 63, P, P, 0, None))
    _refused(q(ctypes.c_void_p(4098), CFR_F32, 4, 64, 64, P, P, 0, None))
    _refused(q(ctypes.c_void_p(4097), CFR_BF16, 4, 64, 64, P, P, 0, None))


def test_mx4_device_ordinal_refused():
    for device in (-1, 4096):
        _refused(load().cfr_mx4_quantize(P, CFR_BF16, 4, 32, 32, P, P, device, None))


def test_mx4_overlaps_refused():
    # 4 x 64 float32 at 4096: 1024 bytes; codes 128 bytes, scales 8
    q, d = load().cfr_mx4_quantize, load().cfr_mx4_dequantize
    far, end = 1 << 20, 4096 + 1024
    for c, s in ((4096, far), (end - 1, far), (far, end - 1), (4096 - 127, far), (far, 4096 - 7)):
        c, s = ctypes.c_void_p(c), ctypes.c_void_p(s)
        for rc in (q(P, CFR_F32, 4, 64, 64, c, s, 4096, None), d(c, s, 4, 64, P, CFR_F32, 64, 4096, None)):
            with pytest.raises(CfrError, match="overlap"):
                check(rc)
    with pytest.raises(CfrError, match="overlap"):
        check(q(P, CFR_F32, 4, 64, 64, ctypes.c_void_p(far), ctypes.c_void_p(far + 127), 4096, None))
    for c, s in ((end, end + 128), (4096 - 128, 4096 - 136), (far, far + 128)):
        with pytest.raises(CfrError, match="device ordinal"):
            check(q(P, CFR_F32, 4, 64, 64, ctypes.c_void_p(c), ctypes.c_void_p(s), 4096, None))


def test_mx4_tensor_checks():
    torch = pytest.importorskip("torch")
    from calibration_free_channel_amd import mx4_dequantize, mx4_quantize
    with pytest.raises(ValueError):
        mx4_quantize(torch.zeros(4, 32))  # not on a device
    with pytest.raises(ValueError):
        mx4_quantize(torch.zeros(4, 32, dtype=torch.int32))
    with pytest.raises(ValueError):
        mx4_dequantize(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8), 32)


def _norm_in(**kw):
    a = dict(x=P, xd=CFR_F32, xs=64, w=None, wd=0, offset=0.0, eps=1e-6, rows=4, cols=64, u=ctypes.c_void_p(1 << 20),
             ud=CFR_F32, us=64, device=0)
    a.update(kw)
    return load().cfr_block_norm_in(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(xd=7), dict(ud=-1), dict(rows=-1), dict(cols=-1), dict(eps=-1.0),
                                 dict(eps=float("nan")), dict(device=-1), dict(device=4096), dict(x=None), dict(u=None),
                                 dict(xs=63), dict(us=10), dict(x=ctypes.c_void_p(4098)),
                                 dict(u=ctypes.c_void_p(4096 + 4)), dict(u=ctypes.c_void_p(4096), us=65),
                                 dict(u=P, ud=CFR_BF16), dict(w=ctypes.c_void_p(1 << 20)),
                                 dict(w=ctypes.c_void_p((1 << 20) + 4 * 3 * 64)), dict(w=P, wd=5)])
def test_norm_in_refusals(bad):
    _refused(_norm_in(**bad))


def test_norm_in_allows_rows_side_by_side():
    # in place, and columns of one buffer, get past the overlap checks to the device's
    for kw in (dict(u=P), dict(xs=128, us=128, u=ctypes.c_void_p(4096 + 4 * 64))):
        with pytest.raises(CfrError, match="device ordinal"):
            check(_norm_in(**kw, device=4096))
    _refused(_norm_in(xs=128, us=128, u=ctypes.c_void_p(4096 + 4 * 63)))
    _refused(_norm_in(xs=128, us=128, u=ctypes.c_void_p(4096 + 4 * 65)))


def test_norm_out_refusals():
    _refused(load().cfr_block_norm_out(None, None))
    for bad in (dict(gate_act=4), dict(rows=-3), dict(eps=-1.0), dict(device=-1), dict(y=0), dict(x=0), dict(x_out=0),
                dict(y_dtype=3), dict(x_dtype=-1), dict(u_out=1 << 22, u_dtype=9, u_stride=64), dict(y_stride=60),
                dict(post_norm=0, post_weight=1 << 23), dict(next_weight=1 << 23), dict(x_out=4096),
                dict(x_out=(1 << 20) + 4), dict(u_out=1 << 21, u_stride=64), dict(u_out=1 << 20, u_stride=64),
                dict(gate=1 << 21, gate_col_stride=1, gate_row_stride=64), dict(gate=1 << 23, gate_row_stride=-1),
                dict(gate=(1 << 23) + 2), dict(post_weight=1 << 21)):
        a = CfrNormOutArgs(y=4096, x=1 << 20, x_out=1 << 21, rows=4, cols=64, y_stride=64, x_stride=64, x_out_stride=64,
                           post_norm=1)
        for k, v in bad.items():
            setattr(a, k, v)
        _refused(load().cfr_block_norm_out(ctypes.byref(a), None))


def test_experts_refusals():
    h = ctypes.c_void_p()
    good = dict(hidden=64, n_experts=4, inter=32, top=2, max_tokens=8, device=0)
    for bad in (dict(hidden=0), dict(hidden=16385), dict(n_experts=0), dict(n_experts=1025), dict(inter=0), dict(inter=16385),
                dict(top=0), dict(top=17), dict(max_tokens=0), dict(max_tokens=65537), dict(device=-1), dict(device=4096)):
        cfg = CfrExpertsConfig(*{**good, **bad}.values())
        _refused(load().cfr_build_experts(ctypes.byref(cfg), P, P, P, P, P, P, None, ctypes.byref(h)))
        assert not h.value
    _refused(load().cfr_build_experts(None, P, P, P, P, P, P, None, ctypes.byref(h)))
    _refused(load().cfr_build_experts(None, P, P, P, P, P, P, None, None))
    _refused(load().cfr_experts_forward(None, P, 0, 64, P, P, 1, P, 64, None))
    _refused(load().cfr_experts_status(None, None))
    load().cfr_experts_free(None)


def test_experts_build_refuses_another_devices_stream():
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace

    from calibration_free_channel_amd import Experts, ExpertsConfig
    with pytest.raises(ValueError, match="stream"):
        Experts.build(ExpertsConfig(64, 4, 32, 2), None, None, None, stream=SimpleNamespace(device=torch.device("cuda", 1)))


def test_tensors_that_need_gradients_are_refused():
    # found before the device is looked at, so that host tensors show it
    torch = pytest.importorskip("torch")
    from calibration_free_channel_amd import block_norm_in, block_norm_out, mx4_dequantize, mx4_quantize
    from calibration_free_channel_amd._ext import ops
    x, g = torch.zeros(4, 32), torch.zeros(4, 32, requires_grad=True)
    codes = torch.zeros(4, 16, dtype=torch.uint8)
    ids = torch.zeros(4, 1, dtype=torch.int32)
    calls = [lambda: block_norm_in(g), lambda: block_norm_out(g, x), lambda: block_norm_out(x, g),
             lambda: ops.experts_forward(None, 32, 1, 0, g, ids, x[:, :1], None),
             lambda: ops.experts_forward(None, 32, 1, 0, x, ids, g[:, :1], None)]
    for call in calls:
        with pytest.raises(ValueError, match="no_grad"):
            call()
        for mode in (torch.no_grad, torch.inference_mode):
            with mode(), pytest.raises(ValueError, match="device"):
                call()
    for call in (lambda: mx4_quantize(g), lambda: mx4_dequantize(codes, codes, 32), lambda: block_norm_in(x)):
        with pytest.raises(ValueError, match="device"):
            call()


def test_negated_views_are_refused():
    # memory that holds the negative of what the tensor stands for
    torch = pytest.importorskip("torch")
    from calibration_free_channel_amd import block_norm_in, block_norm_out, mx4_quantize
    x = torch.zeros(4, 32)
    neg = torch._neg_view(x)
    assert neg.is_neg()
    for call in (lambda: block_norm_in(neg), lambda: block_norm_out(neg, x), lambda: block_norm_out(x, neg), lambda: mx4_quantize(neg)):
        with pytest.raises(ValueError, match="resolve_neg"):
            call()


def test_module_of_another_torch_is_refused():
    torch = pytest.importorskip("torch")
    from calibration_free_channel_amd import _ext
    assert _ext.ops.torch == str(torch.__version__)
    with pytest.raises(RuntimeError, match="build it again"):
        _ext._check_torch("1.0.0", _ext.ops.torch)
