"""The operators around the block beside autograd: they are inference only."""
import pytest

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]

torch = pytest.importorskip("torch")

from calibration_free_channel_amd import (Experts, ExpertsConfig, block_norm_in, block_norm_out, mx4_dequantize,  # noqa: E402
                                          mx4_quantize)


def _calls():
    """Each operator's call on fresh inputs: name -> (call, tensors it reads whose
    gradient would be lost, tensors it writes)."""
    q = [mx4_quantize(torch.randn(s, device="cuda")) for s in ((2, 8, 32), (2, 8, 32), (2, 32, 8))]
    layer = Experts.build(ExpertsConfig(32, 2, 8, 1, 4), *q)
    t = {n: torch.randn(4, 32, device="cuda") for n in ("x", "y", "gate", "out", "next_out")}
    t["weight"], t["next_weight"] = torch.randn(32, device="cuda"), torch.randn(32, device="cuda")
    t["gate_w"], ids = torch.rand(4, 1, device="cuda"), torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    codes, scales = mx4_quantize(t["x"])
    return {
        "quantize": (lambda: mx4_quantize(t["x"], out=(codes, scales)), [], [codes, scales]),
        "dequantize": (lambda: mx4_dequantize(codes, scales, 32, out=t["out"]), [], [t["out"]]),
        "norm_in": (lambda: block_norm_in(t["x"], t["weight"], out=t["out"]), [t["x"], t["weight"]], [t["out"]]),
        "norm_in in place": (lambda: block_norm_in(t["x"], out=t["x"]), [t["x"]], [t["x"]]),
        "norm_out": (lambda: block_norm_out(t["y"], t["x"], post_weight=t["weight"], gate=t["gate"], next_weight=t["next_weight"],
                                            next_norm=True, out=t["out"], next_out=t["next_out"]),
                     [t["y"], t["x"], t["weight"], t["gate"], t["next_weight"]], [t["out"], t["next_out"]]),
        "experts": (lambda: layer.forward(t["x"], ids, t["gate_w"], out=t["out"]), [t["x"], t["gate_w"]], [t["out"]]),
    }


NAMES = ["quantize", "dequantize", "norm_in", "norm_in in place", "norm_out", "experts"]


@pytest.mark.parametrize("name", NAMES)
def test_inputs_that_need_gradients_are_refused(name):
    # the operators have no backward pass, and say so instead of giving results without one
    call, reads, writes = _calls()[name]
    call()
    for t in [*reads, *writes]:
        if not t.is_floating_point():
            continue
        t.requires_grad_(True)
        with pytest.raises(ValueError, match="no_grad"):
            call()
        with torch.no_grad():
            call()
        with torch.inference_mode():
            call()
        t.requires_grad_(False)
    call()


def test_weights_that_need_gradients_are_quantized():
    w = torch.nn.Parameter(torch.randn(4, 32, device="cuda"))
    codes, scales = mx4_quantize(w)  # whole numbers have no gradient
    want = mx4_quantize(w.detach())
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    assert not mx4_dequantize(codes, scales, 32).requires_grad


@pytest.mark.parametrize("name", NAMES)
def test_writes_count_as_changes(name):
    # autograd finds a tensor that it saved changed, as after any in-place operation
    call, _, writes = _calls()[name]
    before = [t._version for t in writes]
    call()
    assert all(t._version == v + 1 for t, v in zip(writes, before))
    a = torch.randn(4, 32, device="cuda", requires_grad=True)
    for out in writes:
        if out.is_floating_point():
            loss = (a * out).sum()  # saves out
            call()
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                loss.backward()


def test_outputs_made_in_inference_mode():
    with torch.inference_mode():
        out = torch.empty(4, 32, device="cuda")
    x = torch.randn(4, 32, device="cuda")
    assert block_norm_in(x, out=out) is out and torch.equal(out, block_norm_in(x))


def test_negated_views_are_refused():
    # memory that holds the negative of what the tensor stands for
    x = torch.randn(4, 32, device="cuda")
    neg = torch._neg_view(x)
    assert neg.is_neg()
    with pytest.raises(ValueError, match="resolve_neg"):
        block_norm_in(neg)
    with pytest.raises(ValueError, match="resolve_neg"):
        block_norm_out(x, neg)
    with pytest.raises(ValueError, match="resolve_neg"):
        mx4_quantize(neg)
    with pytest.raises(ValueError, match="resolve_neg"):
        block_norm_in(x, out=torch._neg_view(torch.empty_like(x)))
    assert torch.equal(block_norm_in(neg.resolve_neg()), -block_norm_in(x))
