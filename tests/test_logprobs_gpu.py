"""Log probabilities of given tokens over logits (flce_token_logprobs and its backward)
against the float64 definitions, at the bounds of head_ops_testlib: types, odd sizes,
strides and alignments, masks that leave few or no ids, equal logits, infinities and NaN
in masked places, temperatures, streams and row offsets past 32 bits."""
import numpy as np
import pytest

import flce_inputs
from head_ops_testlib import check_logprobs, grad_bound
from oracle import head_ops as ho

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _rng(seed):
    return np.random.Generator(np.random.Philox(np.random.SeedSequence([seed, 61])))


def _draw(N, V, seed, dtype, std=2.0):
    z = (_rng(seed).standard_normal((N, V)) * std).astype(np.float32)
    if dtype == "bf16":
        z = flce_inputs.bf16_bits_to_f32(flce_inputs.f32_to_bf16_bits(z))
    return z


def _tokens(N, V, seed, skip=0.2):
    g = _rng(seed + 1000)
    y = g.integers(0, V, N).astype(np.int32)
    y[g.random(N) < skip] = -100
    return y


def _place(z, dtype, pad=0, shift=0):
    """z on the device with row stride V + pad, starting `shift` elements into its memory."""
    N, V = z.shape
    flat = torch.full((shift + N * (V + pad),), 7.0, dtype=TYPES[dtype], device=DEV)
    t = flat[shift:].view(N, V + pad)[:, :V]
    t.copy_(torch.from_numpy(z))
    return t


def _vec(x):
    return None if x is None else torch.from_numpy(np.asarray(x, dtype=np.float32)).to(DEV)


def _run(z, y, dtype, *, top_k=0, T=1.0, pad=0, shift=0, grads="abc", seed=0, ids=True):
    N, V = z.shape
    t = _place(z, dtype, pad, shift)
    tok = None if y is None else torch.from_numpy(y).to(DEV)
    res = flce.token_logprobs(t, tok, top_k=top_k, temperature=T)
    T32 = 1.0 / float(np.float32(1.0) / np.float32(T))
    ref = ho.token_logprobs(z, y, top_k=top_k, temperature=T32)
    check_logprobs(res, ref, z, T32)
    if top_k and ids:
        assert np.array_equal(res.top_id.cpu().numpy(), ref["top_id"])
    if grads:
        g = _rng(seed + 5)
        up = {k: (g.standard_normal(N).astype(np.float32) if k in grads else None) for k in "abc"}
        dz = flce.token_logprobs_backward(t, tok, res, dlogprob=_vec(up["a"]), dentropy=_vec(up["b"]),
                                          dlse=_vec(up["c"]), temperature=T)
        G = ho.token_logprobs_grad(z, y, up["a"], up["b"], up["c"], temperature=T32)
        bound = grad_bound(z, G, ref, up["a"], up["b"], up["c"], T32, TYPES[dtype])
        got = dz.double().cpu().numpy()
        nan = np.isnan(G)
        assert np.array_equal(np.isnan(got), nan)
        over = ~nan & ~(np.abs(got - G) <= bound)
        assert not over.any(), (np.argwhere(over)[:3], np.nanmax(np.abs(got - G) / bound))
        # in place: the same bits
        u = t.clone() if pad == 0 and shift == 0 else _place(z, dtype, pad, shift)
        flce.token_logprobs_backward(u, tok, res, dlogprob=_vec(up["a"]), dentropy=_vec(up["b"]),
                                     dlse=_vec(up["c"]), temperature=T, in_place=True)
        assert torch.equal(torch.nan_to_num(u.float()), torch.nan_to_num(dz.float()))
    return res


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,pad,shift", [
    (1, 1, 0, 0), (1, 2, 3, 1), (3, 7, 0, 0), (5, 33, 0, 3), (2, 1000, 0, 0), (7, 1001, 0, 1),
    (4, 5003, 13, 2), (33, 32000, 0, 0), (9, 32003, 0, 5), (3, 65600, 8, 0), (2, 100003, 0, 7),
    (3, 240007, 1, 3), (300, 257, 0, 0)])
def test_sizes_strides_and_alignments(dtype, N, V, pad, shift):
    z = _draw(N, V, N * 7 + V, dtype)
    _run(z, _tokens(N, V, N + V), dtype, top_k=min(5, V), pad=pad, shift=shift, seed=N)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("top_k", [1, 2, 16, 20, 31, 32])
def test_rankings(dtype, top_k):
    _run(_draw(6, 12345, top_k, dtype), _tokens(6, 12345, 3), dtype, top_k=top_k, grads="")
    _run(_draw(70, 40, top_k, dtype), _tokens(70, 40, 3), dtype, top_k=top_k, grads="")


@pytest.mark.parametrize("T", [0.25, 0.7, 3.0])
def test_temperatures(T):
    for dtype in TYPES:
        _run(_draw(5, 3001, 4, dtype), _tokens(5, 3001, 4), dtype, top_k=4, T=T)


@pytest.mark.parametrize("grads", ["a", "b", "c", "ab"])
def test_single_upstream_gradients(grads):
    _run(_draw(6, 700, 8, "f32"), _tokens(6, 700, 8), "f32", grads=grads)


def test_without_tokens():
    z = _draw(4, 500, 9, "f32")
    r = _run(z, None, "f32", top_k=3, grads="bc")
    assert torch.count_nonzero(r.logprob) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [37, 5003, 70001])
def test_masks(dtype, V):
    """-inf on all ids, on all but one, on all but a few, on most, on the token; the type's
    lowest value in the place of -inf; logits far from 0."""
    lowest = float(torch.finfo(TYPES[dtype]).min)
    z = _draw(10, V, V, dtype)
    y = (np.arange(10) * 3 % V).astype(np.int32)
    g = _rng(V)
    z[0] = -np.inf
    z[1] = -np.inf
    z[1, V - 1] = 2.5
    z[2] = -np.inf
    z[2, [3, 11, V // 2]] = [1.0, 4.0, 1.0]
    z[3, g.random(V) < 0.9] = -np.inf
    z[4, y[4]] = -np.inf
    z[5] = lowest
    z[5, [1, V - 2]] = [0.5, -3.0]
    z[6, : V // 2] = lowest
    z[7] = z[7] + 1024
    z[8] = z[8] - 1024
    y[9] = -100
    z[9] = -np.inf
    if dtype == "bf16":
        z = flce_inputs.bf16_bits_to_f32(flce_inputs.f32_to_bf16_bits(z))
    _run(z, y, dtype, top_k=8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_row_of_the_types_lowest_value(dtype):
    """Uniform in the forward pass, like any constant row; no gradient, as documented."""
    V = 4000
    z = np.full((2, V), float(torch.finfo(TYPES[dtype]).min), dtype=np.float32)
    t = _place(z, dtype)
    tok = torch.tensor([5, -100], dtype=torch.int32, device=DEV)
    r = flce.token_logprobs(t, tok, top_k=3)
    tol = 2.0 ** -22 * 10 * np.log(V)
    assert abs(float(r.entropy[0]) - np.log(V)) < tol and abs(float(r.logprob[0]) + np.log(V)) < tol
    assert r.top_id.tolist() == [[0, 1, 2]] * 2
    assert float((r.top_logprob + np.log(V)).abs().max()) < tol
    ones = torch.ones(2, device=DEV)
    dz = flce.token_logprobs_backward(t, tok, r, dlogprob=ones, dentropy=ones, dlse=ones)
    assert torch.count_nonzero(dz) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [50, 5000, 70000, 300000])
def test_equal_logits_rank_by_id(dtype, V):
    """Constant rows, rows of two values, blocks of large neighbours and signed zeros: more
    ids reach the ranking's threshold than its candidate list holds."""
    z = np.zeros((6, V), dtype=np.float32)
    z[0] = 1.25
    z[1, 1::2] = 1.0
    z[2, V // 3: V // 3 + 40] = 2.0
    z[2, V // 3 + 5] = 3.0
    z[3, ::3] = -0.0
    z[4, -1] = 1.0
    z[5] = -np.arange(V)
    _run(z, _tokens(6, V, 2), dtype, top_k=32, grads="", ids=True) if dtype == "f32" else \
        _run(flce_inputs.bf16_bits_to_f32(flce_inputs.f32_to_bf16_bits(z)), _tokens(6, V, 2), dtype,
             top_k=32, grads="")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [100, 70000])
def test_nan_and_infinity_stay_in_their_rows(dtype, V):
    z = _draw(7, V, 3, dtype)
    y = np.array([0, 1, 2, -100, 4, 5, 6], dtype=np.int32)
    z[0, V // 2] = np.nan
    z[1, V - 1] = np.inf
    z[2, 0] = np.nan
    z[3, 3] = np.inf
    z[4, [1, 2]] = [np.inf, -np.inf]
    z[5, : V // 2] = -np.inf
    _run(z, y, dtype, top_k=4, grads="abc", ids=False)


def test_confident_tokens_keep_their_small_numbers():
    """1 - p down to 1e-30: logprob and the gradient at the token relative to themselves."""
    V = 2000
    z = np.zeros((4, V), dtype=np.float32)
    z[:, 3] = [20.0, 40.0, 60.0, 75.0]
    y = np.full(4, 3, dtype=np.int32)
    r = _run(z, y, "f32", grads="a")
    want = ho.token_logprobs(z, y)["logprob"]
    assert np.all(np.abs(r.logprob.double().cpu().numpy() / want - 1) < 1e-5)


def test_tokens_out_of_range():
    z = _draw(4, 300, 5, "f32")
    y = np.array([1, 300, -1, -100], dtype=np.int32)
    t = _place(z, "f32")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = flce.token_logprobs(t, torch.from_numpy(y).to(DEV), top_k=2, status=status)
    assert flce.check_status(status) == flce.FLCE_ERR_LABEL_RANGE
    assert torch.isnan(r.logprob).tolist() == [False, True, True, False]
    assert torch.isfinite(r.entropy).all() and torch.isfinite(r.top_logprob).all()
    dz = flce.token_logprobs_backward(t, torch.from_numpy(y).to(DEV), r,
                                      dlogprob=torch.ones(4, device=DEV))
    assert torch.isfinite(dz).all() and torch.count_nonzero(dz[1:]) == 0


def test_no_rows():
    t = torch.empty(0, 50, device=DEV)
    y = torch.empty(0, dtype=torch.int32, device=DEV)
    r = flce.token_logprobs(t, y, top_k=3)
    assert r.logprob.shape == (0,) and r.top_id.shape == (0, 3)
    assert flce.token_logprobs_backward(t, y, r, dlogprob=r.logprob).shape == (0, 50)


def test_row_offsets_past_32_bits():
    """70000 rows of 65600 bf16 (9 GB): the last rows start past 2^32 elements."""
    N, V = 70000, 65600
    t = torch.zeros(N, V, dtype=torch.bfloat16, device=DEV)
    z = _draw(3, V, 6, "bf16")
    rows = [0, 33333, N - 1]
    for r, zr in zip(rows, z):
        t[r].copy_(torch.from_numpy(zr))
    y = torch.full((N,), 11, dtype=torch.int32, device=DEV)
    res = flce.token_logprobs(t, y, top_k=3)
    ref = ho.token_logprobs(z, [11] * 3, top_k=3)
    pick = flce.TokenLogprobs(*(getattr(res, k)[rows] for k in
                                ("logprob", "entropy", "lse", "top_logprob", "top_id")))
    check_logprobs(pick, ref, z, 1.0)
    assert np.array_equal(pick.top_id.cpu().numpy(), ref["top_id"])
    a = torch.ones(N, device=DEV)
    flce.token_logprobs_backward(t, y, res, dlogprob=a, in_place=True)
    G = ho.token_logprobs_grad(z, [11] * 3, np.ones(3), None, None)
    got = t[rows].double().cpu().numpy()
    assert np.all(np.abs(got - G) <= grad_bound(z, G, ref, np.ones(3), None, None, 1.0, torch.bfloat16))


def test_repeats_are_bitwise_equal_and_out_is_used():
    z = _draw(40, 32003, 12, "bf16")
    t = _place(z, "bf16")
    y = torch.from_numpy(_tokens(40, 32003, 1)).to(DEV)
    a = flce.token_logprobs(t, y, top_k=8)
    out = {k: torch.empty_like(getattr(a, k)) for k in ("logprob", "entropy", "lse", "top_logprob", "top_id")}
    for _ in range(5):
        b = flce.token_logprobs(t, y, top_k=8, out=out)
        assert b.lse is out["lse"]
        for k in out:
            assert torch.equal(getattr(a, k), out[k]), k


def test_another_stream_and_a_graph():
    z = _draw(64, 50021, 13, "f32")
    y = torch.from_numpy(_tokens(64, 50021, 2)).to(DEV)
    t = _place(z, "f32")
    want = flce.token_logprobs(t, y, top_k=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = flce.token_logprobs(t, y, top_k=8, stream=side)
    r2 = flce.token_logprobs(t, y, top_k=8, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(r.top_id, want.top_id) and torch.equal(r2.lse, want.lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = flce.token_logprobs(t, y, top_k=8)
        d = flce.token_logprobs_backward(t, y, r, dlogprob=r.lse, dentropy=r.lse)
    t.copy_(torch.flip(t, dims=[1]))
    graph.replay()
    torch.cuda.synchronize()
    again = flce.token_logprobs(t, y, top_k=8)
    assert torch.equal(r.top_id, again.top_id) and torch.equal(r.logprob, again.logprob)
    assert torch.equal(d, flce.token_logprobs_backward(t, y, again, dlogprob=again.lse, dentropy=again.lse))


def test_autograd_and_expanded_gradients():
    z = _draw(6, 900, 14, "f32")
    y = _tokens(6, 900, 5)
    t = _place(z, "f32").clone().requires_grad_(True)
    lp, ent, lse = flce.fused_token_logprobs(t.view(2, 3, 900), torch.from_numpy(y).to(DEV).view(2, 3).long())
    assert lp.shape == (2, 3)
    (lp.sum() * 0.5 - ent.mean()).backward()
    G = ho.token_logprobs_grad(z, y, np.full(6, 0.5), np.full(6, -1 / 6), None)
    ref = ho.token_logprobs(z, y)
    bound = grad_bound(z, G, ref, np.full(6, 0.5), np.full(6, 1 / 6), None, 1.0, torch.float32)
    assert np.all(np.abs(t.grad.double().cpu().numpy() - G) <= bound)
