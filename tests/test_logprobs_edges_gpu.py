"""Log probabilities over logits at the edges of their kernels. Bounds count roundings as in
head_ops_testlib, u = 2^-24."""
import math

import numpy as np
import pytest

from head_ops_testlib import U, check_logprobs, sum_eps
from oracle import head_ops as ho

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _rng(seed):
    return np.random.Generator(np.random.Philox(np.random.SeedSequence([seed, 67])))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [0.5, 1.0, 2.0])
def test_gradient_at_a_token_with_the_types_lowest_logit(dtype, T):
    """p is 0 there and 1 - p is 1, whether its log probability still is a number or, at
    temperatures below 1, -inf. At a logit of -inf there is no gradient."""
    lowest = torch.finfo(TYPES[dtype]).min
    z = torch.zeros(3, 40, dtype=TYPES[dtype], device=DEV)
    z[0, 7] = lowest
    z[1, 7] = -math.inf
    z[2, 7] = -1000.0
    y = torch.full((3,), 7, dtype=torch.int32, device=DEV)
    r = flce.token_logprobs(z, y, temperature=T)
    a = torch.tensor([0.75, 0.75, 0.75], device=DEV)
    g = flce.token_logprobs_backward(z, y, r, dlogprob=a, dentropy=a, dlse=a, temperature=T)
    want = torch.tensor([0.75 / T, 0.0, 0.75 / T], device=DEV)
    assert float((g[:, 7].float() - want).abs().max()) <= 4 * U   # 0.75 / T is a number of each type


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 900, 6000, 50000, 240007])
@pytest.mark.parametrize("T", [1.0, 0.7])
def test_rows_with_one_likely_id(dtype, V, T):
    """Where all but one id are masked its log probability is 0 and so is the entropy; where
    the others are merely unlikely, the alternative's log probability is the token's."""
    g = _rng(V)
    top = g.integers(0, V, 40)
    level = (g.standard_normal(40) * 30).astype(np.float32)
    z = torch.full((40, V), -math.inf, device=DEV)
    z[20:] = 0.0
    z += torch.where(torch.isinf(z), 0.0, torch.from_numpy(level).to(DEV)[:, None])
    gap = torch.from_numpy((1 + g.random(40) * 60).astype(np.float32)).to(DEV)
    rows = torch.arange(40, device=DEV)
    z[rows, torch.from_numpy(top).to(DEV)] = torch.from_numpy(level).to(DEV) + gap
    z = z.to(TYPES[dtype])
    tok = torch.from_numpy(top.astype(np.int32)).to(DEV)
    for y in (tok, None):
        r = flce.token_logprobs(z, y, top_k=2, temperature=T)
        assert torch.equal(r.top_id[:, 0], tok)
        assert torch.count_nonzero(r.entropy[:20]) == 0 and bool((r.entropy >= 0).all())
        assert torch.count_nonzero(r.top_logprob[:20, 0]) == 0 and bool((r.top_logprob <= 0).all())
        x = z[rows, tok.long()].double() / T
        assert bool(((r.lse[:20].double() - x[:20]).abs() <= 3 * U * x[:20].abs()).all())
        if y is not None:
            assert torch.count_nonzero(r.logprob[:20]) == 0
            assert torch.equal(r.logprob, r.top_logprob[:, 0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1000, 1003])
def test_the_gradient_takes_no_more_memory_than_its_rows(dtype, V):
    """The last position of each sequence: rows of logits that lie T V elements apart."""
    z = torch.randn(8, 50, V, device=DEV).to(TYPES[dtype])
    y = torch.arange(8, dtype=torch.int32, device=DEV)
    rows = z[:, -1]
    r = flce.token_logprobs(rows, y)
    want = flce.token_logprobs_backward(rows.contiguous(), y, r, dlogprob=r.lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = flce.token_logprobs_backward(rows, y, r, dlogprob=r.lse)
    h = flce.token_logprobs_backward(rows, y, r, dlogprob=r.lse, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for t in (g, h):
        assert t.shape == rows.shape and torch.equal(t, want)
        assert t.untyped_storage().nbytes() <= 8 * (V + 8) * t.element_size() + 16
    leaf = rows.detach().requires_grad_(True)
    lp, _, lse = flce.fused_token_logprobs(leaf, y)
    lp.backward(lse.detach())
    assert torch.equal(leaf.grad, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,pad,skip", [(1003, 0, 1), (1001, 0, 3), (1000, 4, 1), (1002, 3, 2)])
def test_the_gradients_rows_start_as_the_logits_do(dtype, V, pad, skip):
    """Relative to 16 bytes, so that both are accessed 16 bytes at a time."""
    z = torch.randn(9, V + pad, device=DEV).to(TYPES[dtype])[skip:, :V]
    y = torch.arange(9 - skip, dtype=torch.int32, device=DEV)
    r = flce.token_logprobs(z, y)
    g = flce.token_logprobs_backward(z, y, r, dlogprob=r.lse, dentropy=r.lse)
    out = torch.empty(9 - skip, V, dtype=z.dtype, device=DEV)
    flce.token_logprobs_backward(z, y, r, dlogprob=r.lse, dentropy=r.lse, out=out)
    assert torch.equal(g, out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h = flce.token_logprobs_backward(z, y, r, dlogprob=r.lse, dentropy=r.lse, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(g, h)
    for t in (g, h):
        for i in range(9 - skip):
            assert (t[i].data_ptr() - z[i].data_ptr()) % 16 == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,V", [(3, 40, 1000), (2, 100, 64), (5, 4, 504), (1, 20, 304), (4, 1, 80)])
def test_a_shifted_sequence(dtype, B, T, V):
    """logits[:, :-1] with tokens[:, 1:]: the values of a contiguous copy, without making one
    of a long sequence. (Rows start at whole 16 bytes, so that both add up in one order.)"""
    z = torch.randn(B, T + 1, V, device=DEV).to(TYPES[dtype])
    z[:, -1] = math.nan          # the position that is left out counts nowhere
    y = torch.randint(0, V, (B, T + 1), device=DEV)
    y[0, 1] = -100
    up = torch.randn(3, B, T, device=DEV)
    got = []
    for copy in (True, False):
        leaf = z.detach().clone().requires_grad_(True)
        rows = leaf[:, :-1].contiguous() if copy else leaf[:, :-1]
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        out = flce.fused_token_logprobs(rows, y[:, 1:], temperature=0.8)
        spent = torch.cuda.max_memory_allocated() - before
        assert all(t.shape == (B, T) and t.is_contiguous() for t in out)
        if T == 40:
            assert copy or spent < rows.numel() * rows.element_size() // 4
        sum((t * u).sum() for t, u in zip(out, up)).backward()
        got.append([*out, leaf.grad])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    lp, _, _ = flce.fused_token_logprobs(z[:, :-1], None)
    assert torch.count_nonzero(lp) == 0
    with pytest.raises(ValueError):
        flce.fused_token_logprobs(z[:, :-1], y[:, :1].expand(B, T + 1))


def test_other_views_of_logits():
    z = torch.randn(4, 3, 25, 132, device=DEV)
    y = torch.randint(0, 132, (4, 3, 25), device=DEV)
    for cut in (lambda t: t[:, :, 1:], lambda t: t[1:, :2], lambda t: t[:, :, ::2], lambda t: t.transpose(0, 1),
                lambda t: t[:1].expand(4, 3, 25, *t.shape[3:]), lambda t: t[:, :, :24], lambda t: t[:0],
                lambda t: t[:, 1:2, 1:], lambda t: t[:, :, 3], lambda t: t[2, 1, :]):
        got = []
        for copy in (True, False):
            leaf = z.clone().requires_grad_(True)
            rows = cut(leaf)
            lp, ent, lse = flce.fused_token_logprobs(rows.contiguous() if copy else rows, cut(y))
            (lp * 2 + ent - lse * 0.5).sum().backward()
            got.append((lp, ent, lse, leaf.grad))
        for a, b in zip(*got):
            assert torch.equal(a, b)


def _limited(z, y, top_k):
    """token_logprobs with a limit of 1 ns: (outputs by name, status code)."""
    from linear_cross_entropy_flce_gb300 import _ops_binding as B
    N, V = z.shape
    out = {k: torch.zeros(N, device=DEV) for k in ("logprob", "entropy", "lse")}
    if top_k:
        out["top_logprob"] = torch.zeros(N, top_k, device=DEV)
        out["top_id"] = torch.zeros(N, top_k, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    at = {k: t.data_ptr() for k, t in out.items()}
    rc = B._token_logprobs(z.data_ptr(), B._DTYPES[z.dtype], V, y.data_ptr(), N, V,
                           B._options(-100, top_k, 1.0, 0, 1), at["logprob"], at["entropy"], at["lse"],
                           at.get("top_logprob"), at.get("top_id"), status.data_ptr(),
                           torch.cuda.current_stream().cuda_stream)
    assert rc == flce.FLCE_OK
    return out, flce.check_status(status)


@pytest.mark.parametrize("dtype,N,V,sure", [("bf16", 300, 6000, False), ("f32", 2000, 4500, False),
                                            ("bf16", 3, 128256, False), ("bf16", 400, 60000, True),
                                            ("f32", 60, 150000, False), ("f32", 120, 210000, True)])
def test_a_wait_that_runs_out_leaves_nan_and_a_status(dtype, N, V, sure):
    """A 1-ns limit ends every wait that the hardware's own look at the barrier does not (it takes
    a microsecond or so): the call ends, its rows are NaN or right, the status says which, and
    the next call is as ever. With many copies under way some wait does run out."""
    z = torch.randn(N, V, device=DEV).to(TYPES[dtype])
    y = (torch.arange(N, device=DEV) * 7 % V).int()
    ran_out = 0
    for top_k in (0, 5, 0, 5):
        want = flce.token_logprobs(z, y, top_k=top_k)
        out, code = _limited(z, y, top_k)
        late = torch.isnan(out["lse"])
        assert code == (flce.FLCE_ERR_TIMEOUT if bool(late.any()) else flce.FLCE_OK)
        ran_out += code != flce.FLCE_OK
        for k, t in out.items():
            assert torch.equal(t[~late], getattr(want, k)[~late]), k
            if k != "top_id":
                assert bool(torch.isnan(t[late]).all()), k
        again = flce.token_logprobs(z, y, top_k=top_k)
        for k in out:
            assert torch.equal(getattr(again, k), getattr(want, k)), k
    assert ran_out or not sure


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,pad", [(257, 0), (1000, 3), (2003, 0), (4096, 0), (6001, 5), (10007, 0), (24004, 0),
                                   (33000, 0), (60001, 0), (128256, 0), (212900, 4), (240007, 1)])
def test_every_id_counts_once(dtype, V, pad):
    """Row r has the ids r, r + K, r + 2 K, ... at one value and -inf elsewhere, about 64 of them:
    one that is left out or taken twice moves the log-sum-exp by 1 / 64."""
    K = -(-V // 64)
    full = torch.full((K, V + pad), 50.0, dtype=TYPES[dtype], device=DEV)
    z = full[:, :V]
    z.fill_(-math.inf)
    ids = torch.arange(V, device=DEV)
    z[ids % K, ids] = 1.5
    y = torch.arange(K, dtype=torch.int32, device=DEV)
    count = torch.bincount(ids % K, minlength=K).double()
    r = flce.token_logprobs(z, y, top_k=32)
    # the terms are equal: 2^-22 of each, then no more than 65 additions
    e = 2.0 ** -22 + 80 * U
    logn = count.log()
    assert float((r.lse.double() - 1.5 - logn).abs().max()) <= e + 8 * U * 6
    assert float((r.entropy.double() - logn).abs().max()) <= 10 * e
    assert float((r.logprob.double() + logn).abs().max()) <= 4 * e * 5
    k = torch.arange(32, device=DEV)
    want = y[:, None] + K * k[None, :]
    there = want < V
    assert torch.equal(r.top_id, torch.where(there, want, torch.full_like(want, -1)).int())
    assert float((r.top_logprob.double() + logn[:, None])[there].abs().max()) <= 4 * e * 5
    a = torch.ones(K, device=DEV)
    g = flce.token_logprobs_backward(z, y, r, dlogprob=a).double()
    p = torch.zeros_like(g)
    p[ids % K, ids] = 1 / count[ids % K]
    p = -p
    p[y.long(), y.long()] += 1
    half = torch.finfo(TYPES[dtype]).eps / 2
    assert bool(((g - p).abs() <= (half + 64 * U + 4 * e) * p.abs()).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("top_k", [0, 5])
@pytest.mark.parametrize("N,V,threads", [(3000, 6000, 128), (800, 60000, 256), (1300, 3000, 32)])
def test_many_distinct_rows(dtype, top_k, N, V, threads):
    """More rows than CTAs or clusters at once: slots, messages and barriers are used again."""
    t = torch.from_numpy((_rng(N + V).standard_normal((N, V)) * 2).astype(np.float32)).to(DEV).to(TYPES[dtype])
    z = t.float().cpu().numpy()
    y = _rng(N).integers(0, V, N).astype(np.int32)
    y[::7] = -100
    r = flce.token_logprobs(t, torch.from_numpy(y).to(DEV), top_k=top_k)
    ref = ho.token_logprobs(z, y, top_k=top_k)
    check_logprobs(r, ref, z, 1.0, eps=sum_eps(V, threads))
    assert np.array_equal(r.top_id.cpu().numpy() if top_k else ref["top_id"], ref["top_id"])
