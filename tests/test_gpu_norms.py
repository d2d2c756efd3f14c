"""The norms before and after a block on the GPU against the float64 oracle.

Tolerances, before any run.  A sum of squares of n <= 16384 positive terms: a
thread adds at most 16 of them, the wave six times, the workgroup at most 16
partial sums: at most 40 roundings of 2^-24, halved by the square root; three
products, a division and a root after it: below 32 * 2^-24 = 2^-19 relative.
Longer rows add 8 terms per 8192 columns to a thread's chain.  A gate's
activation through the hardware exponential (argument rounded: |z| 2^-24, here
|z| < 8) and reciprocal: below 2^-20.  Rounding to the output's type: half a
step, eps / 2 relative; below the smallest normal the step stops shrinking at
smallest_normal * eps (float16: 2^-14 * 2^-10), so half of that is added."""
import numpy as np
import pytest

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]

torch = pytest.importorskip("torch")

from calibration_free_channel_amd import block_norm_in, block_norm_out  # noqa: E402
from oracle import norms  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF = {t: torch.finfo(t).eps / 2 for t in (F32, BF16, F16)}
TINY = {t: torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2 for t in (F32, BF16, F16)}


def _np(t):
    return t.double().cpu().numpy()


def _rel(cols):
    return 2.0 ** -19 + cols / 8192 * 8 * 2.0 ** -24


def _rand(rows, cols, dtype, seed, pad=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, cols + pad, generator=g) * scale).to(dtype).cuda()[:, :cols]


SIZES = [(1, 1), (3, 2), (1, 8), (5, 7), (2, 31), (9, 64), (1, 128), (33, 511), (4, 512), (7, 520), (2, 1435), (1, 2048),
         (70, 2048), (3, 2049), (2, 4096), (3, 4104), (2, 8192), (2, 8193), (1, 16384), (2, 16383), (2, 16392), (1, 40001)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (F16, F32), (F32, BF16)])
def test_norm_in(rows, cols, dtype, out):
    x = _rand(rows, cols, dtype, rows + cols, pad=(cols % 3) * 8, scale=3.0)
    w = _rand(1, cols, F32, 1)[0].contiguous()
    u = block_norm_in(x, w, eps=1e-5, offset=1.0, dtype=out)
    ref = norms.norm(_np(x), _np(w), 1e-5, 1.0)
    assert u.dtype == out
    assert (np.abs(_np(u) - ref) <= np.abs(ref) * (_rel(cols) + 2.0 ** -23 + HALF[out])
            + np.abs(ref / np.where(_np(w) + 1 == 0, 1, _np(w) + 1)) * 2.0 ** -24 + TINY[out]).all()


@pytest.mark.parametrize("wdtype", [None, F32, BF16, F16])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_norm_in_weights_and_strides(wdtype, pad):
    x = _rand(6, 264, BF16, 3, pad=pad)
    w = None if wdtype is None else _rand(1, 264, wdtype, 4)[0].contiguous()
    wide = torch.full((6, 264 + pad + 3), 5.0, device="cuda")
    u = block_norm_in(x, w, out=wide[:, :264])
    ref = norms.norm(_np(x), None if w is None else _np(w))
    assert (np.abs(_np(u) - ref) <= np.abs(ref) * (_rel(264) + HALF[F32])).all()
    assert (wide[:, 264:] == 5).all()


def test_norm_in_place_three_dimensions_and_empty():
    x = _rand(12, 96, F32, 5).contiguous().view(3, 4, 96)
    ref = norms.norm(_np(x))
    assert block_norm_in(x, out=x) is x
    assert (np.abs(_np(x) - ref) <= np.abs(ref) * 2.0 ** -18).all()
    assert block_norm_in(torch.empty(0, 64).cuda()).shape == (0, 64)
    assert block_norm_in(torch.empty(4, 0).cuda()).shape == (4, 0)


def test_rows_do_not_meet():
    # a NaN, an infinity and a row of zeros leave the other rows exact
    x = _rand(8, 512, F32, 6)
    clean = _np(block_norm_in(x))
    x[1, 3], x[4, 0], x[6] = float("nan"), float("inf"), 0.0
    u = _np(block_norm_in(x))
    for r in (0, 2, 3, 5, 7):
        np.testing.assert_array_equal(u[r], clean[r])
    assert np.isnan(u[1]).all() and np.isnan(u[4, 0]) and (u[4, 1:] == 0).all() and (u[6] == 0).all()
    assert np.isnan(_np(block_norm_in(x, eps=0.0))[6]).all()  # 0 / 0, as the formula


def _check_out(y, x, **kw):
    rows, cols = y.shape
    nxt = kw.pop("next_norm", True)
    got = block_norm_out(y, x, next_norm=nxt, **kw)
    s, u = got if nxt else (got, None)
    ref = {k: (_np(v) if isinstance(v, torch.Tensor) else v) for k, v in kw.items()
           if k not in ("out", "next_out", "next_dtype", "stream")}
    v, rs, ru = norms.norm_out(_np(y), _np(x), **ref)
    tol = np.abs(v) * (_rel(cols) + 2.0 ** -18) + (np.abs(v) + np.abs(rs - v)) * 2.0 ** -22
    assert s.dtype == x.dtype
    assert (np.abs(_np(s) - rs) <= tol + np.abs(rs) * HALF[x.dtype] + TINY[x.dtype]).all()
    if nxt:
        ms = np.sqrt(np.mean(rs * rs, -1, keepdims=True) + kw.get("eps", 1e-6))
        off = np.sqrt(np.mean(tol * tol, -1, keepdims=True)) / ms
        f = 1.0 if kw.get("next_weight") is None else np.abs(_np(kw["next_weight"])) + abs(kw.get("offset", 0.0))
        want = np.abs(ru) * (off + _rel(cols) + HALF[u.dtype]) + (tol + np.abs(rs) * 2.0 ** -23) / ms * f
        assert (np.abs(_np(u) - ru) <= want + TINY[u.dtype]).all()
    return s, u


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("yd,xd", [(BF16, F32), (BF16, BF16), (F32, F32), (F16, BF16)])
def test_norm_out(rows, cols, yd, xd):
    y, x = _rand(rows, cols, yd, 2 * rows + cols, scale=4.0), _rand(rows, cols, xd, 7, scale=2.0)
    g = _rand(rows, cols, yd, 8)
    _check_out(y, x, post_weight=_rand(1, cols, F32, 9)[0].contiguous(), gate=g, gate_act="silu", out_scale=0.5,
               resid_scale=1.25, next_weight=_rand(1, cols, F32, 10)[0].contiguous(), offset=1.0)


@pytest.mark.parametrize("gate", ["none", "token", "channel", "full", "wide", "every other"])
@pytest.mark.parametrize("act", ["none", "sigmoid", "silu", "tanh"])
@pytest.mark.parametrize("post,nxt", [(True, True), (True, False), (False, True), (False, False)])
def test_norm_out_gates(gate, act, post, nxt):
    rows, cols = 37, 1032
    y, x = _rand(rows, cols, BF16, 11), _rand(rows, cols, F32, 12)
    g = {"none": lambda: None, "token": lambda: _rand(rows, 1, BF16, 13), "channel": lambda: _rand(1, cols, BF16, 13),
         "full": lambda: _rand(rows, cols, BF16, 13), "wide": lambda: _rand(rows, cols, BF16, 13, pad=3),
         "every other": lambda: _rand(rows, 2 * cols, BF16, 13)[:, ::2]}[gate]()
    _check_out(y, x, post_norm=post, gate=g, gate_act=act, next_norm=nxt)


def test_many_rows_per_workgroup():
    # more rows than workgroups, at one, two and four waves' sums per row
    for rows, cols in ((9000, 72), (5000, 600), (3000, 2056)):
        y, x = _rand(rows, cols, BF16, 14), _rand(rows, cols, BF16, 15)
        for post, nxt in ((True, True), (False, True), (True, False)):
            _check_out(y, x, post_norm=post, next_norm=nxt)


def test_in_place_residual_and_channel_gate_vector():
    y, x = _rand(6, 256, BF16, 16).contiguous(), _rand(6, 256, F32, 17).contiguous()
    want, _ = _check_out(y, x.clone(), gate=torch.tensor([[0.5]], dtype=BF16).cuda())
    s, u = block_norm_out(y, x, gate=torch.tensor([[0.5]], dtype=BF16).cuda(), next_norm=True, out=x)
    assert s is x and torch.equal(x, want)
    for cols in (256, 20000):  # long rows too
        y, x = _rand(3, cols, F32, 18).contiguous(), _rand(3, cols, F32, 19).contiguous()
        g = _rand(1, cols, F32, 20)[0].contiguous()
        want, wu = block_norm_out(y, x, gate=g, gate_act="tanh", next_norm=True)
        s, u = block_norm_out(y, x, gate=g, gate_act="tanh", next_norm=True, out=x)
        assert torch.equal(x, want) and torch.equal(u, wu)


def test_rows_of_one_buffer_side_by_side():
    # block output, residual and result as columns of one wide buffer
    buf = torch.randn(9, 4 * 128).cuda()
    y, x, o, u = (buf[:, i * 128:(i + 1) * 128] for i in range(4))
    want, wu = block_norm_out(y.clone(), x.clone(), next_norm=True)
    block_norm_out(y, x, next_norm=True, out=o, next_out=u)
    assert torch.equal(o, want) and torch.equal(u, wu)


def test_large_gate_arguments():
    z = torch.tensor([[-1e4, -100.0, -88.5, 88.5, 100.0, 1e4, 0.0, -0.0]]).cuda()
    y, x = torch.ones(1, 8).cuda(), torch.zeros(1, 8).cuda()
    for act in ("sigmoid", "silu", "tanh"):
        s = _np(block_norm_out(y, x, post_norm=False, gate=z, gate_act=act))
        np.testing.assert_allclose(s, norms.act(_np(z), act), rtol=1e-5, atol=1e-30)


def test_graph_replay_and_own_stream():
    y, x = _rand(64, 512, BF16, 21).contiguous(), _rand(64, 512, F32, 22).contiguous()
    out, nxt = torch.empty_like(x), torch.empty_like(y)
    block_norm_out(y, x, next_norm=True, out=out, next_out=nxt)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block_norm_out(y, x, next_norm=True, out=out, next_out=nxt)
    for seed in range(3):
        y.copy_(_rand(64, 512, BF16, 30 + seed))
        g.replay()
        torch.cuda.synchronize()
        a, b = block_norm_out(y, x, next_norm=True)
        assert torch.equal(a, out) and torch.equal(b, nxt)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = block_norm_out(y, x, next_norm=True, stream=s)
    c = block_norm_in(x, stream=s)
    s.synchronize()
    assert torch.equal(a, out) and torch.equal(b, nxt) and torch.equal(c, block_norm_in(x))


def test_overlaps_are_refused():
    x = torch.randn(8, 64).cuda()
    with pytest.raises(RuntimeError):
        block_norm_in(x[:4], out=x[2:6])
    with pytest.raises(RuntimeError):
        block_norm_out(x[:4], x[4:], out=x[:4])
    with pytest.raises(RuntimeError):
        block_norm_out(x[:4], x[4:], next_norm=True, next_out=x[4:])


@pytest.mark.parametrize("lead", [(), (3,), (2, 3)])
def test_rows_without_columns(lead):
    y, x = torch.zeros(*lead, 0, dtype=BF16).cuda(), torch.zeros(*lead, 0).cuda()
    for gate in (torch.zeros(0, dtype=BF16), torch.zeros(*lead, 0, dtype=BF16), torch.zeros(1, dtype=BF16)):
        s, u = block_norm_out(y, x, gate=gate.cuda(), next_norm=True)
        assert s.shape == u.shape == x.shape and s.dtype == F32 and u.dtype == BF16
    assert block_norm_in(x).shape == x.shape


@pytest.mark.parametrize("shape,gate", [((1, 1), ()), ((6, 40), ()), ((6, 40), (40,)), ((6, 40), (1, 40)), ((2, 3, 40), (2, 3, 1)),
                                        ((2, 3, 40), (2, 3, 40)), ((40,), (40,)), ((40,), (1,)), ((6, 1), (6, 1))])
def test_gate_shapes(shape, gate):
    # without norms, x = 0 and y = 1 the result is the gate as it is
    y, x, g = torch.ones(shape).cuda(), torch.zeros(shape).cuda(), torch.randn(gate).cuda()
    assert torch.equal(block_norm_out(y, x, post_norm=False, gate=g), g.expand(shape))
    if y.dim() < 3:
        with pytest.raises(ValueError):
            block_norm_out(y, x, post_norm=False, gate=torch.randn(2, 7).cuda())


@pytest.mark.parametrize("shape,gate,as_shape", [
    ((2, 3, 40), (3, 2, 40), None), ((2, 3, 40), (6, 1, 40), None), ((2, 3, 40), (3, 2, 1), None), ((2, 3, 40), (1, 6, 1), None),
    ((2, 3, 40), (6, 1), None), ((2, 3, 40), (6, 40), None), ((2, 3, 40), (1, 3, 40), None), ((2, 3, 40), (2, 1, 40), None),
    ((2, 3, 40), (3, 1), None), ((2, 2, 40), (2, 40), None), ((6, 40), (2, 3, 40), None), ((6, 40), (2, 3, 1), None),
    ((2, 3, 40), (1, 1, 40), (1, 1, 40)), ((2, 3, 40), (1, 40), (1, 1, 40)), ((2, 3, 40), (40,), (1, 1, 40)),
    ((2, 3, 40), (1, 1, 1), (1, 1, 1)), ((2, 3, 40), (1, 2, 3, 1), (2, 3, 1)), ((1, 6, 40), (6, 1), (1, 6, 1)),
    ((1, 6, 40), (6, 40), (1, 6, 40)), ((6, 40), (1, 6, 40), (6, 40)), ((2, 1, 1, 40), (2, 1, 1, 1), (2, 1, 1, 1))])
def test_gate_rows_are_the_tokens(shape, gate, as_shape):
    # a gate has one row, or y's rows: the same leading sizes, ones before them
    # aside, not only as many.  as_shape: how it broadcasts, None: it is refused
    y, x, g = torch.ones(shape).cuda(), torch.zeros(shape).cuda(), torch.randn(gate).cuda()
    if as_shape is None:
        with pytest.raises(ValueError, match="broadcast"):
            block_norm_out(y, x, post_norm=False, gate=g)
    else:
        assert torch.equal(block_norm_out(y, x, post_norm=False, gate=g), g.view(as_shape).expand(shape))
