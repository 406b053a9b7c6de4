"""Log probabilities straight from hidden states (flce_linear_token_logprobs and its
backward) against the float64 definitions. Hidden states and weights lie on grids on
which every logit is exact in fp32, so that the rankings have one right answer."""
import numpy as np
import pytest

from head_ops_testlib import U, check_logprobs, half_step
from oracle import head_ops as ho

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"


def _rng(seed):
    return np.random.Generator(np.random.Philox(np.random.SeedSequence([seed, 62])))


def _inputs(N, D, V, seed, h_std=1.0, w_std=None):
    """float64 H, W on grids of 2^-5 and 2^-11 with at most 8 significant bits."""
    g = _rng(seed)
    w_std = w_std if w_std is not None else 1.3 / np.sqrt(D)
    H = np.clip(np.round(g.standard_normal((N, D)) * 32 * h_std), -255, 255) / 32
    W = np.clip(np.round(g.standard_normal((V, D)) * 2048 * w_std), -255, 255) / 2048
    y = g.integers(0, V, N).astype(np.int32)
    y[g.random(N) < 0.15] = -100
    return H, W, y


def _dev(x, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV).to(dtype)


def _vec(x):
    return None if x is None else torch.from_numpy(np.asarray(x, dtype=np.float32)).to(DEV)


def _check_grads(H, W, y, up, T, dH, dW):
    """Each G entry is rounded once to bf16 (2^-8) after fp32 errors of 1e-5 or so; the fp32
    sums of K products add 2^-22 sqrt(K) of their magnitude; then the output's rounding."""
    Z = H @ W.T
    G = ho.token_logprobs_grad(Z, y, *up, temperature=T)
    rho = 2.0 ** -8 + 1e-4
    for got, A, B, K in ((dH, G, W, W.shape[0]), (dW, G.T, H, H.shape[0])):
        if got is None:
            continue
        want, size = A @ B, np.abs(A) @ np.abs(B)
        bound = (rho + 2.0 ** -22 * np.sqrt(K)) * size + half_step(got.dtype) * np.abs(want) * 1.01 + 1e-30
        err = np.abs(got.double().cpu().numpy() - want)
        assert np.all(err <= bound), float(np.max(err / bound))


def _run(N, D, V, seed, *, top_k=0, T=1.0, grads=True, dw_dtype="float32", **kw):
    H, W, y = _inputs(N, D, V, seed, **kw)
    Hd, Wd, yd = _dev(H), _dev(W), torch.from_numpy(y).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = flce.linear_token_logprobs(Hd, Wd, yd, top_k=top_k, temperature=T, status=status)
    assert flce.check_status(status) == flce.FLCE_OK
    T32 = 1.0 / float(np.float32(1.0) / np.float32(T))
    Z = H @ W.T
    ref = ho.token_logprobs(Z, y, top_k=top_k, temperature=T32)
    check_logprobs(r, ref, Z, T32, eps=U * (V // 4 + 64) + 2.0 ** -20)
    if top_k:
        assert np.array_equal(r.top_id.cpu().numpy(), ref["top_id"])
    if grads:
        g = _rng(seed + 3)
        up = [g.standard_normal(N).astype(np.float32) / N for _ in range(3)]
        dH, dW = flce.linear_token_logprobs_backward(
            Hd, Wd, yd, r, dlogprob=_vec(up[0]), dentropy=_vec(up[1]), dlse=_vec(up[2]),
            temperature=T, dw_dtype=dw_dtype, status=status)
        assert flce.check_status(status) == flce.FLCE_OK
        _check_grads(H, W, y, up, T32, dH, dW)
    return r


@pytest.mark.parametrize("N,D,V", [
    (1, 8, 1), (1, 64, 5), (2, 128, 256), (1, 512, 5003), (3, 200, 257), (5, 64, 33000), (16, 256, 3001),
    (17, 512, 4096), (64, 1000, 2000), (127, 128, 1000), (128, 136, 1100), (129, 256, 9999),
    (255, 64, 700), (257, 512, 1500), (700, 256, 3000)])
def test_shapes(N, D, V):
    _run(N, D, V, N + D + V, top_k=min(V, 5), dw_dtype="bfloat16" if N % 2 else "float32")


@pytest.mark.parametrize("N", [1, 40, 200])
@pytest.mark.parametrize("top_k", [1, 8, 20, 32])
def test_rankings(N, top_k):
    _run(N, 64, 7000, 11 * top_k + N, top_k=top_k, grads=False)


@pytest.mark.parametrize("T", [0.5, 2.0])
def test_temperatures(T):
    _run(30, 128, 2000, 4, top_k=4, T=T)


def test_peaked_rows():
    _run(60, 256, 3000, 5, top_k=6, h_std=2.0, w_std=0.1)


def test_equal_weight_rows_rank_by_id():
    """W rows in groups of equal ones, and all equal: ties across tiles and ranges."""
    for V, rep in ((4000, 4000), (4000, 16), (1000, 2)):
        H, W, y = _inputs(9, 64, V // rep, V + rep)
        W = np.tile(W, (rep, 1))
        y = np.zeros(9, dtype=np.int32)
        r = flce.linear_token_logprobs(_dev(H), _dev(W), torch.from_numpy(y).to(DEV), top_k=32)
        ref = ho.token_logprobs(H @ W.T, y, top_k=32)
        assert np.array_equal(r.top_id.cpu().numpy(), ref["top_id"])


def test_ragged_vocabulary_with_very_negative_logits():
    """Padded columns are zeros in the tile and must not beat the logits, all below -60."""
    N, D, V = 10, 64, 300
    g = _rng(9)
    H = np.ones((N, D))
    W = -(np.round(g.random((V, D)) * 100) + 28) / 64
    y = np.arange(N).astype(np.int32)
    r = flce.linear_token_logprobs(_dev(H), _dev(W), torch.from_numpy(y).to(DEV), top_k=5)
    ref = ho.token_logprobs(H @ W.T, y, top_k=5)
    check_logprobs(r, ref, H @ W.T, 1.0, eps=U * (V // 4 + 64) + 2.0 ** -20)
    assert np.array_equal(r.top_id.cpu().numpy(), ref["top_id"])


def test_nan_in_one_hidden_state_stays_in_its_row():
    H, W, y = _inputs(20, 64, 1000, 10)
    y[:] = 3
    H[4, 7] = np.nan
    Hd, Wd = _dev(H), _dev(W)
    r = flce.linear_token_logprobs(Hd, Wd, torch.from_numpy(y).to(DEV), top_k=3)
    bad = torch.zeros(20, dtype=torch.bool, device=DEV)
    bad[4] = True
    assert torch.equal(torch.isnan(r.logprob), bad) and torch.equal(torch.isnan(r.lse), bad)
    assert torch.equal(torch.isnan(r.top_logprob).all(1), bad)


def test_without_tokens_and_out_of_range():
    H, W, _ = _inputs(6, 64, 500, 12)
    Hd, Wd = _dev(H), _dev(W)
    r = flce.linear_token_logprobs(Hd, Wd, None, top_k=2)
    assert torch.count_nonzero(r.logprob) == 0
    dH, dW = flce.linear_token_logprobs_backward(Hd, Wd, None, r, dentropy=torch.ones(6, device=DEV))
    _check_grads(H, W, None, (None, np.ones(6), None), 1.0, dH, dW)
    y = torch.tensor([0, 500, -7, 499, -100, 3], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = flce.linear_token_logprobs(Hd, Wd, y, status=status)
    assert flce.check_status(status) == flce.FLCE_ERR_LABEL_RANGE
    assert torch.isnan(r.logprob).tolist() == [False, True, True, False, False, False]


def test_requested_gradients_only_and_no_rows():
    H, W, y = _inputs(30, 64, 600, 13)
    Hd, Wd, yd = _dev(H), _dev(W), torch.from_numpy(y).to(DEV)
    r = flce.linear_token_logprobs(Hd, Wd, yd)
    a = _rng(1).standard_normal(30).astype(np.float32)
    both = flce.linear_token_logprobs_backward(Hd, Wd, yd, r, dlogprob=_vec(a))
    dH, none = flce.linear_token_logprobs_backward(Hd, Wd, yd, r, dlogprob=_vec(a), need_dw=False)
    assert none is None and torch.equal(dH, both[0])
    none, dW = flce.linear_token_logprobs_backward(Hd, Wd, yd, r, dlogprob=_vec(a), need_dh=False)
    assert none is None and torch.equal(dW, both[1])
    r0 = flce.linear_token_logprobs(Hd[:0], Wd, yd[:0], top_k=2)
    dH, dW = flce.linear_token_logprobs_backward(Hd[:0], Wd, yd[:0], r0, dlogprob=r0.logprob)
    assert dH.shape == (0, 64) and torch.count_nonzero(dW) == 0


def test_cross_entropy_is_the_negative_mean():
    """a = -1 / n reproduces the loss gradient of the fused cross-entropy of the same head."""
    H, W, y = _inputs(300, 256, 3000, 14)
    Hd, Wd, yd = _dev(H), _dev(W), torch.from_numpy(y).to(DEV)
    n = int((y != -100).sum())
    r = flce.linear_token_logprobs(Hd, Wd, yd)
    ce = flce.forward_backward(Hd, Wd, yd)
    assert abs(float(-r.logprob.sum() / n) - float(ce.loss)) <= 1e-5 * float(ce.loss)
    dH, dW = flce.linear_token_logprobs_backward(Hd, Wd, yd, r,
                                                 dlogprob=torch.full((300,), -1.0 / n, device=DEV))
    for got, want in ((dH, ce.dH), (dW, ce.dW)):
        got, want = got.double(), want.double()
        # two roundings of each G entry to bf16, or of its fp32 value's neighbour
        assert float((got - want).norm() / want.norm()) <= 2.0 ** -7


def test_several_blocks_and_chunks():
    """20000 ids make two vocabulary chunks: dH is accumulated over them."""
    _run(300, 64, 20000, 15, dw_dtype="float32")
    _run(300, 64, 20000, 16, dw_dtype="bfloat16")


def test_repeats_streams_and_graphs():
    H, W, y = _inputs(50, 128, 9000, 17)
    Hd, Wd, yd = _dev(H), _dev(W), torch.from_numpy(y).to(DEV)
    want = flce.linear_token_logprobs(Hd, Wd, yd, top_k=8)
    a = _vec(_rng(3).standard_normal(50))
    g0 = flce.linear_token_logprobs_backward(Hd, Wd, yd, want, dlogprob=a, dentropy=a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = flce.linear_token_logprobs(Hd, Wd, yd, top_k=8, stream=side)
    g1 = flce.linear_token_logprobs_backward(Hd, Wd, yd, r, dlogprob=a, dentropy=a, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for k in ("logprob", "entropy", "lse", "top_logprob", "top_id"):
        assert torch.equal(getattr(r, k), getattr(want, k)), k
    assert torch.equal(g0[0], g1[0]) and torch.equal(g0[1], g1[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = flce.linear_token_logprobs(Hd, Wd, yd, top_k=8)
        g1 = flce.linear_token_logprobs_backward(Hd, Wd, yd, r, dlogprob=a, dentropy=a)
    Hd.copy_(torch.flip(Hd, dims=[0]))
    graph.replay()
    torch.cuda.synchronize()
    again = flce.linear_token_logprobs(Hd, Wd, yd, top_k=8)
    assert torch.equal(r.top_id, again.top_id) and torch.equal(r.entropy, again.entropy)


def test_autograd():
    H, W, y = _inputs(24, 128, 2000, 18)
    Hd, Wd = _dev(H).view(2, 12, 128).requires_grad_(True), _dev(W).requires_grad_(True)
    lp, ent, lse = flce.fused_linear_token_logprobs(Hd, Wd, torch.from_numpy(y).to(DEV).view(2, 12))
    (lp.sum() + 0.1 * ent.sum()).backward()
    _check_grads(H, W, y, (np.ones(24), np.full(24, np.float32(0.1)), None), 1.0,
                 Hd.grad.view(24, 128), Wd.grad)


@pytest.mark.parametrize("top_k", [1, 7, 32])
@pytest.mark.parametrize("N,V,high", [(300, 20000, 2), (700, 9000, 3), (129, 50000, 1), (2500, 70000, 2)])
def test_equal_logits_of_many_tokens_rank_by_id(N, V, high, top_k):
    # whole-number products, exact in fp32: rows full of ties, over and around 0
    g = np.random.Generator(np.random.Philox(np.random.SeedSequence([N + V, 64])))
    H = g.integers(-high, high + 1, (N, 16)).astype(np.float64)
    W = g.integers(-high, high + 1, (V, 16)).astype(np.float64)
    H[5] = 0.0
    H[6] = np.abs(H[6]) * -40
    W[V // 2:] = W[:V - V // 2]   # every logit comes twice
    Z = H @ W.T
    order = np.argsort(-Z, axis=1, kind="stable")[:, :top_k]
    runs = []
    for _ in range(3):
        r = flce.linear_token_logprobs(_dev(H), _dev(W), None, top_k=top_k)
        runs.append(r.top_id.cpu().numpy())
        assert np.array_equal(runs[-1], order)
