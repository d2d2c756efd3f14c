"""The routed experts on microscaled 4-bit weights against the float64 oracle.

Tolerances come from oracle.experts.tolerance: h is rounded to bfloat16
(2^-8) for bfloat16 tokens in calls of more than 64 slots, to 16 bits (2^-16)
below and for float16, to 24 bits (2^-24) for float32."""
import numpy as np
import pytest

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]

torch = pytest.importorskip("torch")

from calibration_free_channel_amd import Experts, ExpertsConfig, mx4_dequantize, mx4_quantize  # noqa: E402
from calibration_free_channel_amd._lib import CfrError  # noqa: E402
from oracle import experts as oracle  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
DTYPES = [BF16, F16, F32]


class Layer:
    def __init__(self, H, E, I, top, max_tokens, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.H, self.E, self.I, self.top = H, E, I, top
        mats = [torch.randn(E, r, c, generator=g) * 2.0 / c ** 0.5 for r, c in ((I, H), (I, H), (H, I))]
        self.q = [mx4_quantize(m.cuda()) for m in mats]
        self.np = [tuple(t.cpu().numpy() for t in p) for p in self.q]
        self.ex = Experts.build(ExpertsConfig(H, E, I, top, max_tokens), *self.q)

    def tokens(self, T, dtype, seed=1, pad=0, empty=0.0, hot=None):
        g = torch.Generator().manual_seed(seed)
        x = torch.randn(T, self.H + pad, generator=g)
        ids = torch.stack([torch.randperm(self.E, generator=g)[:self.top] for _ in range(T)]).int()
        if hot is not None:
            ids[:, 0] = hot  # may repeat an expert within a token
        ids[torch.rand(T, self.top, generator=g) < empty] = -1
        w = torch.rand(T, self.top, generator=g)
        return x.to(dtype).cuda()[:, :self.H], ids.cuda(), w.cuda()

    def check(self, x, ids, w, y):
        T, dt = x.shape[0], x.dtype
        fi = torch.finfo(dt)
        h_half = {F32: 2.0 ** -24, F16: 2.0 ** -16, BF16: 2.0 ** -8 if T * self.top > 64 else 2.0 ** -16}[dt]
        ref, parts, spread = oracle.forward(x.double().cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy(), *self.np, bounds=True)
        tol = oracle.tolerance(ref, parts, spread, self.H, self.top * self.I, h_half, fi.eps / 2,
                               fi.smallest_normal * fi.eps / 2)
        got = y.double().cpu().numpy()
        assert y.dtype == dt and np.isfinite(got).all()
        worst = np.max(np.abs(got - ref) / tol)
        assert worst <= 1, worst
        assert (got[(ids.cpu().numpy() < 0).all(1)] == 0).all()


# hidden, experts, inter, top
SHAPES = [(256, 16, 64, 2), (1, 1, 1, 1), (31, 2, 17, 2), (33, 3, 33, 1), (128, 5, 40, 5), (264, 7, 300, 3), (640, 130, 24, 16),
          (2048, 8, 768, 8), (300, 65, 257, 4)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_oracle(shape, dtype):
    layer = Layer(*shape, max_tokens=150)
    top = shape[3]
    few = 64 // top  # the largest call on the path for few slots, and the smallest beyond it
    for T in sorted({1, 2, min(few, 150), min(few + 1, 150), 150}):
        x, ids, w = layer.tokens(T, dtype, seed=T)
        layer.check(x, ids, w, layer.ex.forward(x, ids, w))
    assert layer.ex.status() == 0
    layer.ex.close()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [5, 32, 33, 300])
def test_strides_and_odd_alignment(dtype, T):
    layer = Layer(96, 4, 32, 2, max_tokens=300)
    for pad in (1, 8):
        x, ids, w = layer.tokens(T, dtype, pad=pad)
        wide = torch.full((T, 96 + pad), 3.0, dtype=dtype, device="cuda")
        layer.ex.forward(x, ids, w, out=wide[:, :96])
        layer.check(x, ids, w, wide[:, :96])
        assert (wide[:, 96:] == 3).all()
    layer.ex.close()


@pytest.mark.parametrize("dtype", DTYPES)
def test_full_tiles_of_one_expert(dtype):
    # one expert takes a slot of every token: tiles of 32, 64 and 128 slots, whole and with one slot more or less
    layer = Layer(256, 4, 96, 2, max_tokens=700)
    for T in (31, 32, 33, 63, 64, 65, 127, 128, 129, 257, 700):
        x, ids, w = layer.tokens(T, dtype, seed=T, hot=3)
        layer.check(x, ids, w, layer.ex.forward(x, ids, w))
    layer.ex.close()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [6, 90, 400])
def test_empty_slots_and_ids_beyond(dtype, T):
    layer = Layer(256, 16, 64, 4, max_tokens=400)
    x, ids, w = layer.tokens(T, dtype, empty=0.5)
    ids[0], ids[T - 1] = -1, -7
    w[ids < 0] = float("nan")  # not read
    y = layer.ex.forward(x, ids, w)
    layer.check(x, ids, torch.nan_to_num(w), y)
    assert layer.ex.status() == 0
    far = ids.clone()
    far[1, 2], far[2, 0] = 16, 2 ** 31 - 1
    want = ids.clone()
    want[1, 2], want[2, 0] = -1, -1
    assert torch.equal(layer.ex.forward(x, far, torch.nan_to_num(w)), layer.ex.forward(x, want, torch.nan_to_num(w)))
    assert layer.ex.status() == 1 and layer.ex.status() == 0
    ids.fill_(-1)
    assert (layer.ex.forward(x, ids, w) == 0).all()
    layer.ex.close()


@pytest.mark.parametrize("T", [3, 100])
def test_nan_stays_in_its_token(T):
    for dtype in DTYPES:
        layer = Layer(256, 8, 64, 2, max_tokens=100)
        x, ids, w = layer.tokens(T, dtype)
        clean = layer.ex.forward(x, ids, w)
        x[1, 7] = float("nan")
        x[2, 9] = float("inf")
        y = layer.ex.forward(x, ids, w)
        keep = [t for t in range(T) if t not in (1, 2)]
        assert torch.equal(y[keep], clean[keep])
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
        layer.ex.close()


def test_large_and_tiny_tokens():
    # activations far from one, within what float32 sums hold
    layer = Layer(256, 4, 64, 2, max_tokens=80)
    for T in (4, 80):
        for scale in (1e-12, 1e4, 1e9):
            x, ids, w = layer.tokens(T, F32)
            x = x * scale
            layer.check(x, ids, w, layer.ex.forward(x, ids, w))
    layer.ex.close()


def test_deterministic_and_independent_of_other_tokens():
    layer = Layer(512, 32, 128, 4, max_tokens=500)
    x, ids, w = layer.tokens(500, BF16)
    y = layer.ex.forward(x, ids, w)
    for _ in range(5):
        assert torch.equal(layer.ex.forward(x, ids, w), y)
    perm = torch.randperm(500).cuda()
    z = layer.ex.forward(x[perm].contiguous(), ids[perm].contiguous(), w[perm].contiguous())
    assert torch.equal(z, y[perm])
    layer.ex.close()


def test_calls_of_changing_size_share_a_workspace():
    layer = Layer(256, 16, 64, 2, max_tokens=300)
    for T in (300, 1, 33, 200, 2, 64, 299):
        for dtype in DTYPES:
            x, ids, w = layer.tokens(T, dtype, seed=T, empty=0.2)
            layer.check(x, ids, w, layer.ex.forward(x, ids, w))
    assert layer.ex.forward(x[:0], ids[:0], w[:0]).shape == (0, 256)
    layer.ex.close()


@pytest.mark.parametrize("T", [4, 120])
def test_graph_replay_and_own_stream(T):
    layer = Layer(256, 16, 64, 4, max_tokens=120)
    x, ids, w = layer.tokens(T, BF16)
    out = layer.ex.forward(x, ids, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = layer.ex.forward(x, ids, w, stream=s)
    s.synchronize()
    assert torch.equal(y, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.ex.forward(x, ids, w, out=out)
    for seed in range(4):
        a, b, c = layer.tokens(T, BF16, seed=seed + 50, empty=0.1 * seed)
        x.copy_(a), ids.copy_(b), w.copy_(c)
        g.replay()
        torch.cuda.synchronize()
        layer.check(x, ids, w, out)
        assert torch.equal(layer.ex.forward(x, ids, w), out)  # eager work between the replays
    layer.ex.close()


def test_odd_columns_ignore_the_unused_half_byte():
    layer = Layer(33, 2, 17, 1, max_tokens=4)
    x, ids, w = layer.tokens(4, F32)
    y = layer.ex.forward(x, ids, w)
    dirty = []
    for (c, s), cols in zip(layer.q, (33, 33, 17)):
        c = c.clone()
        c[..., -1] |= 0x70
        dirty.append((c, s))
    other = Experts.build(ExpertsConfig(33, 2, 17, 1, 4), *dirty)
    assert torch.equal(other.forward(x, ids, w), y)
    other.close()
    layer.ex.close()


def test_refusals():
    layer = Layer(64, 4, 32, 2, max_tokens=8)
    x, ids, w = layer.tokens(8, BF16)
    bad_scale = (layer.q[0][0], torch.full_like(layer.q[0][1], 255))
    with pytest.raises(CfrError):
        Experts.build(layer.ex.cfg, bad_scale, layer.q[1], layer.q[2])
    with pytest.raises(ValueError):
        Experts.build(layer.ex.cfg, layer.q[2], layer.q[1], layer.q[2])
    with pytest.raises(CfrError):
        layer.ex.forward(torch.cat([x, x]), torch.cat([ids, ids]), torch.cat([w, w]))  # above max_tokens
    with pytest.raises(CfrError):
        layer.ex.forward(x, ids, w, out=x)
    for a in ((x.double(), ids, w), (x[:, :32], ids, w), (x, ids.long(), w), (x, ids[:4], w), (x, ids, w.double()),
              (x.cpu(), ids, w), (x, ids, w.cpu())):
        with pytest.raises(ValueError):
            layer.ex.forward(*a)
    layer.ex.close()
    with pytest.raises(CfrError):
        layer.ex.forward(x, ids, w)


@pytest.mark.parametrize("shape,T", [((16384, 3, 40, 2), 3), ((16384, 3, 40, 2), 40), ((48, 2, 16384, 2), 3), ((48, 2, 16384, 2), 40),
                                     ((64, 1024, 32, 16), 4), ((64, 1024, 32, 16), 70)])
def test_largest_shapes(shape, T):
    layer = Layer(*shape, max_tokens=T)
    for dtype in DTYPES:
        x, ids, w = layer.tokens(T, dtype)
        layer.check(x, ids, w, layer.ex.forward(x, ids, w))
    layer.ex.close()


def test_most_tokens_and_slots():
    # 65536 tokens of 16 slots: a million slots, most of them one expert's; the
    # first and last tokens and some between against the oracle, and every token
    # against the same token in a small call of the same path
    layer = Layer(64, 5, 32, 16, max_tokens=65536)
    T = 65536
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, 64, generator=g).to(BF16).cuda()
    ids = torch.randint(-1, 5, (T, 16), generator=g).int()
    ids[:, 3:] = 2  # the same expert many times in one token
    ids, w = ids.cuda(), torch.rand(T, 16, generator=g).cuda()
    y = layer.ex.forward(x, ids, w)
    for at in (0, 777, 32768, T - 40):
        s = slice(at, at + 40)
        layer.check(x[s], ids[s], w[s], y[s])
    layer.ex.close()


def test_rows_further_apart_than_32_bits_of_bytes():
    layer = Layer(256, 4, 64, 4, max_tokens=20)
    step = (1 << 28) + 256  # 20 rows of bfloat16: 10.7 GB
    buf = torch.zeros(19 * step + (128 << 20) + 256, dtype=BF16, device="cuda")
    for T in (10, 20):  # both paths
        x, ids, w = layer.tokens(T, BF16)
        far = torch.as_strided(buf, (T, 256), (step, 1))
        far.copy_(x)
        y = layer.ex.forward(far, ids, w)
        assert torch.equal(y, layer.ex.forward(x, ids, w))
        out = torch.as_strided(buf, (T, 256), (step, 1), 128 << 20)
        layer.ex.forward(x, ids, w, out=out)
        assert torch.equal(out, y)
    layer.ex.close()


def test_two_layers_at_once_on_two_streams():
    a, b = Layer(256, 16, 64, 4, max_tokens=300, seed=1), Layer(512, 8, 128, 2, max_tokens=300, seed=2)
    xa, xb = a.tokens(300, BF16), b.tokens(300, F16)
    ya, yb = a.ex.forward(*xa), b.ex.forward(*xb)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append((a.ex.forward(*xa, stream=sa), b.ex.forward(*xb, stream=sb)))
    torch.cuda.synchronize()
    for p, q in got:
        assert torch.equal(p, ya) and torch.equal(q, yb)
    a.ex.close()
    b.ex.close()


def test_two_graphs_of_one_layer_one_after_the_other():
    layer = Layer(256, 16, 64, 4, max_tokens=120)
    small, large = layer.tokens(4, BF16), layer.tokens(120, F16, seed=9)
    want = [layer.ex.forward(*small), layer.ex.forward(*large)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for args in (small, large):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer.ex.forward(*args))
        graphs.append(g)
    for order in ((0, 1), (1, 0), (1, 1, 0, 0)):
        for o in outs:
            o.zero_()
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    layer.ex.close()


@pytest.mark.parametrize("T", [8, 70])
def test_tokens_and_output_side_by_side_in_one_buffer(T):
    layer = Layer(64, 4, 32, 2, max_tokens=T)
    x, ids, w = layer.tokens(T, BF16)
    both = torch.full((T, 2 * 64), 7.0, dtype=BF16, device="cuda")
    both[:, :64] = x
    layer.ex.forward(both[:, :64], ids, w, out=both[:, 64:])
    assert torch.equal(both[:, :64], x) and torch.equal(both[:, 64:], layer.ex.forward(x, ids, w))


def test_output_over_an_input_is_refused():
    layer = Layer(64, 4, 32, 2, max_tokens=8)
    x, ids, w = layer.tokens(8, F32)
    buf = torch.zeros(9 * 64, device="cuda")
    for out in (x, torch.as_strided(x, (4, 64), (64, 1), 32)):
        with pytest.raises(CfrError):
            layer.ex.forward(x[: len(out)], ids[: len(out)], w[: len(out)], out=out)
    out = buf[: 8 * 64].view(8, 64)
    with pytest.raises(CfrError):
        layer.ex.forward(x, ids, buf[500:516].view(8, 2), out=out)
    with pytest.raises(CfrError):
        layer.ex.forward(x, buf.view(torch.int32)[:16].view(8, 2), w, out=out)
    layer.ex.forward(x, ids, buf[8 * 64 : 8 * 64 + 16].view(8, 2), out=out)


def _one_channel_layer(d, E=2, top=2, max_tokens=300):
    """Experts with one channel in use: G reads x[0] times 64, V reads x[1], and
    d [E, H] is the channel's column of D.  With x[0] = 1, silu(64) is 64 to
    float32's last bit, so h = 64 x[1] is exact in bfloat16 and a slot's value
    is w d h up to float32 rounding."""
    H = d.shape[1]
    G, V, D = torch.zeros(E, 4, H), torch.zeros(E, 4, H), torch.zeros(E, H, 4)
    G[:, 0, 0], V[:, 0, 1], D[:, :, 0] = 64.0, 1.0, torch.from_numpy(d).float()
    q = [mx4_quantize(m.cuda()) for m in (G, V, D)]
    assert torch.equal(mx4_dequantize(*q[2], 4).cpu(), D)  # d is made of values the format holds
    return Experts.build(ExpertsConfig(H, E, 4, top, max_tokens), *q)


def _one_channel_tokens(T, H, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.zeros(T, H)
    x[:, 0], x[:, 1] = 1.0, (1.0 + torch.rand(T, generator=g)) * torch.sign(torch.randn(T, generator=g))
    return x.to(BF16), g


@pytest.mark.parametrize("T", [40, 150, 300])  # tiles of 32, 64 and 128 slots
@pytest.mark.parametrize("spread", [1, 14, 40])
@pytest.mark.parametrize("shift", [-118, -60, 0, 70])
def test_slots_products_of_bfloat16_prompts(T, spread, shift):
    """What a slot's values keep between the product and the sum over the
    slots.  Rows of D of sizes 2^0 .. 2^(spread - 1) side by side, and two slots
    that nearly cancel, so that y's own rounding hides nothing.  Each value is
    rounded to float16 (2^-11 of it) after scaling that puts the largest of its
    64 at 2^14 or above, where half a step of the smallest float16 numbers,
    2^-25, is 2^-39 of that largest.  To that come the float32 roundings of w d h
    and of the sum, 3 * 2^-24 of the values, and y's rounding, 2^-8 of y."""
    H = 256
    rng = np.random.default_rng(spread + T)
    d = rng.choice([1.0, -1.5], (2, H)) * np.exp2(rng.integers(0, spread, H))
    ex = _one_channel_layer(d)
    x, g = _one_channel_tokens(T, H, seed=T)
    u = 1.0 + torch.rand(T, generator=g)
    w = torch.stack([u, -u * (1 + 2.0 ** -6 * torch.rand(T, generator=g))], 1) * 2.0 ** shift
    ids = torch.tensor([[0, 1]]).repeat(T, 1).int()
    y = ex.forward(x.cuda(), ids.cuda(), w.cuda()).double().cpu().numpy()
    v = w.double().numpy()[:, :, None] * d[None] * (64 * x.double().numpy()[:, 1])[:, None, None]  # [T, slot, H]
    ref = v.sum(1)
    top = np.abs(v).reshape(T, 2, H // 64, 64).max(3).repeat(64, 2)
    tol = (np.abs(v) * (2.0 ** -11 + 3 * 2.0 ** -24) + 2.0 ** -39 * top).sum(1) + np.abs(ref) * 2.0 ** -8
    tiny = 2.0 ** -126 * 2.0 ** -7 / 2 + 2 * 2.0 ** -126 * 2.0 ** -23  # denormal steps of y and of the slots' values
    off = np.abs(y - ref) / (tol * (1 + 2.0 ** -7) + tiny)
    assert off.max() <= 1, off.max()
    ex.close()


@pytest.mark.parametrize("T", [20, 40, 150, 300])  # 20: the path of few slots, which the others agree with
def test_infinity_in_one_column_leaves_the_others(T):
    # a value beyond float32 in one column of one slot: that column is infinite,
    # and its neighbours keep what they would have without it
    H = 128
    rng = np.random.default_rng(T)
    d = rng.choice([1.0, -1.5], (2, H)) * np.exp2(rng.integers(0, 6, (2, H)))
    d[0, 5] = 2.0 ** 121
    ex = _one_channel_layer(d)
    x, g = _one_channel_tokens(T, H, seed=T)
    w = 4.0 + torch.rand(T, 2, generator=g)
    ids = torch.tensor([[0, 1]]).repeat(T, 1).int()
    y = ex.forward(x.cuda(), ids.cuda(), w.cuda()).double().cpu().numpy()
    h = 64 * x.double().numpy()[:, 1]
    v = w.double().numpy()[:, :, None] * d[None] * h[:, None, None]
    assert (y[:, 5] == np.sign(h) * np.inf).all()
    keep = [c for c in range(H) if c != 5]
    ref = v.sum(1)[:, keep]
    tol = np.abs(v).sum(1)[:, keep] * (2.0 ** -11 + 3 * 2.0 ** -24 + 2.0 ** -39 * 2 ** 6) + np.abs(ref) * 2.0 ** -8
    assert (np.abs(y[:, keep] - ref) <= tol * (1 + 2.0 ** -7)).all()
    ex.close()


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_token_of_the_largest_call(dtype):
    # a million slots: each token as it comes out of calls a thirty-second as
    # large, which take the same tiles; a token's result does not depend on its
    # place, so they are equal bit for bit
    layer = Layer(64, 5, 32, 16, max_tokens=65536)
    T, part = 65536, 2048
    g = torch.Generator().manual_seed(4)
    x = torch.randn(T, 64, generator=g).to(dtype).cuda()
    ids = torch.randint(-1, 5, (T, 16), generator=g).int()
    ids[:, 5:] = 2  # most slots are one expert's
    ids, w = ids.cuda(), torch.rand(T, 16, generator=g).cuda()
    y = layer.ex.forward(x, ids, w)
    for at in range(0, T, part):
        s = slice(at, at + part)
        assert torch.equal(layer.ex.forward(x[s], ids[s], w[s]), y[s]), at
    for at in (1000, 50000):
        s = slice(at, at + 40)
        layer.check(x[s], ids[s], w[s], y[s])
    layer.ex.close()


def test_status_after_status():
    # the flag of a call made right after the last status(), on a stream of its own, is not lost
    layer = Layer(64, 4, 32, 2, max_tokens=40)
    s = torch.cuda.Stream()
    for T in (2, 40):
        x, ids, w = layer.tokens(T, BF16)
        ids[T - 1, 0] = 4
        torch.cuda.synchronize()
        for _ in range(50):
            layer.ex.forward(x, ids, w, stream=s)
            assert layer.ex.status() == 1
    assert layer.ex.status() == 0
    layer.ex.close()


@pytest.mark.parametrize("T", [40, 150, 300])
def test_tokens_of_very_different_size_in_one_tile(T):
    # routing weights of 0, of 2^-120 and ones that carry one column past float32, and
    # tokens whose h is zero or tiny, between ordinary ones: each token's values
    # have powers of two of their own
    H = 128
    rng = np.random.default_rng(T)
    d = rng.choice([1.0, -1.5], (2, H)) * np.exp2(rng.integers(0, 6, (2, H)))
    d[0, 5] = 2.0 ** 70
    ex = _one_channel_layer(d)
    x, g = _one_channel_tokens(T, H, seed=T)
    scale = torch.tensor([1.0, 2.0 ** 60, 0.0, 2.0 ** -120, 1.0, 2.0 ** 30])[torch.randint(0, 6, (T,), generator=g)]
    x[:, 1] *= torch.tensor([1.0, 1.0, 0.0, 2.0 ** -100])[torch.randint(0, 4, (T,), generator=g)]
    w = scale[:, None] * (1.0 + torch.rand(T, 2, generator=g))
    ids = torch.tensor([[0, 1]]).repeat(T, 1).int()
    y = ex.forward(x.cuda(), ids.cuda(), w.cuda()).double().cpu().numpy()
    v = w.double().numpy()[:, :, None] * d[None] * (64 * x.double().numpy()[:, 1])[:, None, None]
    past = np.abs(v) >= 2.0 ** 128
    assert past.any() and (past.sum(1)[:, [c for c in range(H) if c != 5]] == 0).all()
    ref = np.where(past, np.copysign(np.inf, v), v).sum(1)
    kept = np.where(past, 0.0, v)
    top = np.abs(kept).reshape(T, 2, H // 64, 64).max(3).repeat(64, 2)
    with np.errstate(invalid="ignore"):
        tol = (np.abs(kept) * (2.0 ** -11 + 3 * 2.0 ** -24) + 2.0 ** -39 * top).sum(1) + np.abs(ref) * 2.0 ** -8
        ok = (y == ref) | (np.abs(y - ref) <= tol * (1 + 2.0 ** -7) + 2.0 ** -126)
    # a y of float32 below 2^128 may round up to bfloat16's infinity: none here is as near
    assert ok.all(), np.argwhere(~ok)[:5]
    ex.close()


@pytest.mark.parametrize("T", [4, 40])
def test_misaligned_pointers_are_refused(T):
    from calibration_free_channel_amd._lib import CFR_F32, check, load
    layer = Layer(64, 4, 32, 2, max_tokens=T)
    x, ids, w = layer.tokens(T, F32)
    y = torch.zeros_like(x)
    good = [x.data_ptr(), ids.data_ptr(), w.data_ptr(), y.data_ptr()]
    for k, off in ((0, 2), (1, 2), (1, 1), (2, 2), (3, 2)):
        a = list(good)
        a[k] += off
        with pytest.raises(CfrError, match="aligned"):
            check(load().cfr_experts_forward(layer.ex._h, a[0], CFR_F32, 64, a[1], a[2], T, a[3], 64, None))
    torch.cuda.synchronize()
    assert (y == 0).all()
    layer.ex.close()
