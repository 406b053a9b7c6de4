"""Log probabilities from hidden states at the edges of their kernels. Bounds count roundings as
in head_ops_testlib, u = 2^-24."""
import math

import numpy as np
import pytest

from head_ops_testlib import U
from oracle import head_ops as ho

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"


@pytest.mark.parametrize("N", [5, 100, 200, 700])
@pytest.mark.parametrize("top_k", [0, 6])
def test_ids_masked_through_the_weight(N, top_k):
    """The last hidden value is 1 and the weight's last column 0, or -inf for ids that cannot
    come: logits of -inf, as over given logits. One row's ids are all masked."""
    D, V = 64, 3001
    g = np.random.Generator(np.random.Philox(np.random.SeedSequence([N, 68])))
    H = np.clip(np.round(g.standard_normal((N, D)) * 32), -255, 255) / 32
    W = np.clip(np.round(g.standard_normal((V, D)) * 300), -255, 255) / 2048
    H[:, -1], W[:, -1] = 1.0, 0.0
    dead = g.random(V) < 0.3
    dead[:300] = True
    dead[-40:] = True
    y = g.integers(0, V, N).astype(np.int32)
    y[:2] = 5                       # a masked token
    Z = H @ W.T
    Z[:, dead] = -np.inf
    W[dead, -1] = -np.inf
    Hd, Wd = torch.from_numpy(H).to(DEV).bfloat16(), torch.from_numpy(W).to(DEV).bfloat16()
    yd = torch.from_numpy(y).to(DEV)
    r = flce.linear_token_logprobs(Hd, Wd, yd, top_k=top_k)
    ref = ho.token_logprobs(Z, y, top_k=top_k)
    for name in ("logprob", "entropy", "lse"):
        got, want = getattr(r, name).double().cpu().numpy(), ref[name]
        inf = np.isinf(want)
        assert np.array_equal(got[inf], want[inf]), name
        assert np.all(np.abs(got[~inf] - want[~inf]) <= 4 * (2.0 ** -22 + U * 200) * 10), name
    if top_k:
        assert np.array_equal(r.top_id.cpu().numpy(), ref["top_id"])
    a = g.standard_normal((3, N)).astype(np.float32)
    up = [torch.from_numpy(t).to(DEV) for t in a]
    dH, dW = flce.linear_token_logprobs_backward(Hd, Wd, yd, r, dlogprob=up[0], dentropy=up[1], dlse=up[2])
    G = ho.token_logprobs_grad(Z, y, *a)
    rho = 2.0 ** -8 + 1e-4
    want, size = G.T @ H, np.abs(G).T @ np.abs(H)
    assert np.all(np.abs(dW.double().cpu().numpy() - want) <= (rho + 2.0 ** -20) * size + 1e-30)
    Wf = W[:, :-1]
    want, size = G @ Wf, np.abs(G) @ np.abs(Wf)     # the last column meets -inf
    got = dH.double().cpu().numpy()[:, :-1]
    assert np.all(np.abs(got - want) <= (rho + 2.0 ** -20) * size + 2.0 ** -8 * np.abs(want) + 1e-30)


def test_rows_whose_every_id_is_masked():
    for N in (3, 150):
        H = torch.zeros(N, 64, device=DEV)
        H[:, -1] = 1.0
        W = torch.zeros(1001, 64, device=DEV)
        W[:, -1] = -math.inf
        y = torch.arange(N, dtype=torch.int32, device=DEV)
        y[0] = -100
        r = flce.linear_token_logprobs(H.bfloat16(), W.bfloat16(), y, top_k=3)
        assert bool((r.lse == -math.inf).all()) and torch.count_nonzero(r.entropy) == 0
        assert bool((r.logprob[1:] == -math.inf).all()) and float(r.logprob[0]) == 0
        assert bool((r.top_id == -1).all()) and bool((r.top_logprob == -math.inf).all())


@pytest.mark.parametrize("N", [7, 300])
def test_rows_with_one_likely_id(N):
    """A token far above the others: its log probability as an alternative is the token's, and
    with the others below 2^-150 of it both are 0, and so is the entropy."""
    D, V = 64, 5000
    H = torch.zeros(N, D, device=DEV)
    H[torch.arange(N), torch.arange(N) % 32] = 1.0
    W = torch.zeros(V, D, device=DEV)
    ids = torch.arange(32, device=DEV) * 150 + 3
    W[ids, torch.arange(32, device=DEV)] = torch.arange(32, device=DEV) * 8.0 + 11.0
    H, W = H.bfloat16(), W.bfloat16()
    y = ids[torch.arange(N, device=DEV) % 32].int()
    for tok in (y, None):
        r = flce.linear_token_logprobs(H, W, tok, top_k=3, temperature=0.75)
        far = (torch.arange(N, device=DEV) % 32) * 8 + 11 > 120
        assert torch.equal(r.top_id[:, 0], y)
        assert bool((r.top_logprob <= 0).all()) and torch.count_nonzero(r.top_logprob[far, 0]) == 0
        assert torch.count_nonzero(r.entropy[far]) == 0
        if tok is not None:
            assert torch.equal(r.logprob, r.top_logprob[:, 0])


@pytest.mark.parametrize("N,D,V,sure", [(3, 512, 33000, True), (100, 1024, 20000, True), (200, 512, 33000, True),
                                        (700, 1024, 9000, True), (40, 64, 300, False)])
def test_a_wait_that_runs_out_leaves_nan(N, D, V, sure):
    """A 1-ns limit: the calls end, what they did not compute is NaN, with a status word or
    without, the status says so, and the next calls are as ever."""
    g = torch.Generator(device=DEV)
    g.manual_seed(N)
    H = torch.randn(N, D, generator=g, device=DEV).bfloat16()
    W = (torch.randn(V, D, generator=g, device=DEV) * 0.05).bfloat16()
    y = (torch.arange(N, device=DEV) * 11 % V).int()
    up = torch.randn(N, generator=g, device=DEV)

    def same_or_nan(got, want):
        return bool((torch.isnan(got) | (got == want)).all())

    ran_out = [0, 0]
    for top_k in (0, 5, 0, 5):
        want = flce.linear_token_logprobs(H, W, y, top_k=top_k)
        for status in (torch.zeros(1, dtype=torch.int32, device=DEV), None):
            r = flce.linear_token_logprobs(H, W, y, top_k=top_k, timeout_ns=1, status=status)
            late = torch.isnan(r.lse)
            for k in ("logprob", "entropy", "lse") + (("top_logprob",) if top_k else ()):
                got, right = getattr(r, k), getattr(want, k)
                assert torch.equal(got[~late], right[~late]) and bool(torch.isnan(got[late]).all()), k
            if status is not None:
                code = flce.check_status(status)
                assert code in (flce.FLCE_OK, flce.FLCE_ERR_TIMEOUT)
                assert code == flce.FLCE_ERR_TIMEOUT or not bool(late.any())
                ran_out[0] += bool(late.any())
        again = flce.linear_token_logprobs(H, W, y, top_k=top_k)
        assert torch.equal(again.lse, want.lse) and torch.equal(again.logprob, want.logprob)
    for dtype in ("float32", "bfloat16"):
        right = flce.linear_token_logprobs_backward(H, W, y, want, dlogprob=up, dentropy=up, dw_dtype=dtype)
        for need in ((True, True), (True, False), (False, True)):
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            got = flce.linear_token_logprobs_backward(
                H, W, y, want, dlogprob=up, dentropy=up, dw_dtype=dtype, need_dh=need[0], need_dw=need[1],
                timeout_ns=1, status=status)
            code = flce.check_status(status)
            nan = any(bool(torch.isnan(t).any()) for t in got if t is not None)
            assert code == (flce.FLCE_ERR_TIMEOUT if nan else flce.FLCE_OK)
            assert all(same_or_nan(t, w) for t, w in zip(got, right) if t is not None)
            ran_out[1] += nan
        again = flce.linear_token_logprobs_backward(H, W, y, want, dlogprob=up, dentropy=up, dw_dtype=dtype)
        assert torch.equal(again[0], right[0]) and torch.equal(again[1], right[1])
    assert min(ran_out) > 0 or not sure


def _classes(N, V, D=64):
    """H and W whose logits are 0 where id and row agree mod D, and -128 elsewhere."""
    H = torch.zeros(N, D, device=DEV)
    H[torch.arange(N, device=DEV), torch.arange(N, device=DEV) % D] = 1.0
    W = torch.full((V, D), -128.0, device=DEV)
    W[torch.arange(V, device=DEV), torch.arange(V, device=DEV) % D] = 0.0
    return H.bfloat16(), W.bfloat16()


@pytest.mark.parametrize("top_k", [0, 32])
@pytest.mark.parametrize("N,V", [(3, 1000), (40, 4099), (128, 9001), (129, 4099), (200, 33000), (300, 16640),
                                 (2500, 7013)])
def test_every_id_counts_once(N, V, top_k):
    """Each row has V / 64 ids that count: one left out or taken twice moves its log-sum-exp by
    64 / V, 500 times the bound or more."""
    H, W = _classes(N, V)
    cls = torch.arange(N, device=DEV) % 64
    y = cls.int()
    count = ((V - 1 - cls) // 64 + 1).double()
    r = flce.linear_token_logprobs(H, W, y, top_k=top_k)
    e = 2.0 ** -22 + U * (16 + 8)   # ones, whose sums are exact, joined by powers of 2
    logn = count.log()
    assert float((r.lse.double() - logn).abs().max()) <= e + 4 * U * 8
    assert float((r.entropy.double() - logn).abs().max()) <= 16 * e
    assert float((r.logprob.double() + logn).abs().max()) <= 4 * e * 8
    if top_k:
        k = torch.arange(32, device=DEV)
        want = cls[:, None] + 64 * k[None, :]
        there = want < V
        assert torch.equal(r.top_id[there], want[there].int())
    dH, dW = flce.linear_token_logprobs_backward(H, W, y, r, dlse=torch.ones(N, device=DEV))
    # dlse: G = p. dW's row v sums p of its class's rows of H; G is rounded to bf16
    rows = torch.bincount(cls, minlength=64).double()
    p = 1 / ((V - 1 - torch.arange(64, device=DEV)) // 64 + 1).double()
    ids = torch.arange(V, device=DEV)
    want = torch.zeros(V, 64, dtype=torch.float64, device=DEV)
    want[ids, ids % 64] = (rows * p)[ids % 64]
    assert bool(((dW.double() - want).abs() <= (2.0 ** -8 + 1e-4) * want).all())
