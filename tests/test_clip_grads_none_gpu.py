"""Parameters without a gradient among those that are clipped."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"


def test_a_missing_gradient_is_passed_over():
    a, b = torch.full((300,), 3.0, device=DEV), torch.full((7, 100), -4.0, device=DEV).bfloat16()
    want = flce.grad_norm([a, b])
    assert torch.equal(flce.grad_norm([None, a, None, b]), want)
    outs = [None, torch.empty_like(a), torch.empty_like(a), torch.empty_like(b)]
    assert torch.equal(flce.clip_grads([None, a, None, b], 1.0, out=outs), want)
    frozen = torch.nn.Linear(4, 4, device=DEV).requires_grad_(False)
    assert torch.equal(flce.clip_grads([a, *(p.grad for p in frozen.parameters()), b], 1.0), want)
    assert torch.equal(a, outs[1]) and torch.equal(b, outs[3])
    assert float(flce.clip_grads([None, None], 1.0)) == 0.0 and float(flce.grad_norm([None])) == 0.0


def test_out_still_needs_a_tensor_for_each():
    a = torch.ones(8, device=DEV)
    with pytest.raises(ValueError):
        flce.clip_grads([a, None], 1.0, out=[torch.empty_like(a)])
    with pytest.raises(ValueError):
        flce.clip_grads([a, a], 1.0, out=[torch.empty_like(a)])
