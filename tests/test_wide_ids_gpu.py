"""64-bit ids that 32 bits do not hold are out of range, not the ids of their low 32 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"
LEAST, MOST = -2 ** 31, 2 ** 31 - 1
FAR = [2 ** 32 + 5, 2 ** 32 - 100, -2 ** 32 + 7, 2 ** 31, LEAST - 1, 2 ** 62, -2 ** 63]


@pytest.mark.parametrize("ignore", [-100, -1, LEAST, MOST, 5])
def test_embedding(ignore):
    W = torch.randn(10, 8, device=DEV, requires_grad=True)
    t = torch.tensor([3, 5, ignore, *FAR, 9], device=DEV)
    y = flce.fused_embedding(t, W, ignore_index=ignore)
    bad = torch.tensor([False] * 3 + [True] * len(FAR) + [False], device=DEV)
    assert torch.equal(y.isnan().all(1), bad) and torch.equal(y.isnan().any(1), bad)
    assert torch.equal(y[0], W[3]) and torch.equal(y[-1], W[9]) and bool((y[2] == 0).all())
    y.backward(torch.ones_like(y))
    want = torch.zeros(10, 8, device=DEV)
    want[[3, 5, 9]] = 1
    if ignore == 5:
        want[5] = 0
    assert torch.equal(W.grad, want)


@pytest.mark.parametrize("ignore", [-100, LEAST, MOST])
def test_log_probabilities(ignore):
    z = torch.randn(2 + len(FAR), 40, device=DEV)
    t = torch.tensor([3, ignore, *FAR], device=DEV)
    lp, _, _ = flce.fused_token_logprobs(z, t, ignore_index=ignore)
    assert lp.isnan().tolist() == [False, False] + [True] * len(FAR) and float(lp[1]) == 0
    H, W = torch.randn(2 + len(FAR), 64, device=DEV).bfloat16(), torch.randn(40, 64, device=DEV).bfloat16()
    lp, _, _ = flce.fused_linear_token_logprobs(H, W, t, ignore_index=ignore)
    assert lp.isnan().tolist() == [False, False] + [True] * len(FAR) and float(lp[1]) == 0


def test_loss_is_that_of_ids_out_of_range():
    H, W = torch.randn(2 + len(FAR), 64, device=DEV).bfloat16(), torch.randn(40, 64, device=DEV).bfloat16()
    t = torch.tensor([3, -100, *FAR], device=DEV)
    out = torch.where((t < 40) & (t >= -100), t, torch.full_like(t, -1)).int()
    a, b = flce.fused_linear_cross_entropy(H, W, t), flce.fused_linear_cross_entropy(H, W, out)
    assert torch.equal(a.nan_to_num(9.0), b.nan_to_num(9.0))


def test_narrow_and_wrong_types():
    W = torch.randn(10, 8)
    t = torch.tensor([[3], [9]])
    for dtype in (torch.uint8, torch.int8, torch.int16, torch.uint32, torch.int64):
        y = flce.fused_embedding(t.to(dtype).to(DEV), W.to(DEV))
        assert torch.equal(y.cpu(), W.index_select(0, t.flatten()).view(2, 1, 8))
    with pytest.raises(TypeError):
        flce.fused_embedding(torch.tensor([3.0], device=DEV), W.to(DEV))


@pytest.mark.parametrize("ignore", [2 ** 32 + 3, 2 ** 31, LEAST - 1])
def test_ignore_index_past_32_bits_is_refused(ignore):
    """2^32 + 3 is not the id 3."""
    W, z = torch.randn(10, 64, device=DEV), torch.randn(2, 10, device=DEV)
    t = torch.tensor([3, 4], dtype=torch.int32, device=DEV)
    H = torch.randn(2, 64, device=DEV).bfloat16()
    for call in (
            lambda: flce.embedding(W, t, ignore_index=ignore), lambda: flce.fused_embedding(t, W, ignore_index=ignore),
            lambda: flce.embedding_backward(torch.ones(2, 64, device=DEV), t, 10, ignore_index=ignore),
            lambda: flce.token_logprobs(z, t, ignore_index=ignore),
            lambda: flce.linear_token_logprobs(H, W.bfloat16(), t, ignore_index=ignore),
            lambda: flce.forward(H, W.bfloat16(), t, ignore_index=ignore)):
        with pytest.raises(ValueError):
            call()
