"""Embedding lookup and the gradient of its table against the float64 definitions.

Bounds, u = 2^-24: a looked-up element is one product and one rounding to its type. A row of the
gradient adds up at most `range` values in a row, then parts of up to `ranges` ranges, every
eighth one by the same thread, then eight: u (range + ranges / 8 + 12) of the sum of magnitudes;
the scale, and the old value where it is added to, are two more roundings, and the type's one."""
import numpy as np
import pytest

from head_ops_testlib import U, half_step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _matrix(rows, D, dtype, seed, pad=0, shift=0):
    """[rows, D] with row stride D + pad from element `shift` of a larger buffer, and that buffer."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    flat = torch.randn(shift + rows * (D + pad) + 8, generator=g, device=DEV).to(TYPES[dtype])
    return flat[shift:shift + rows * (D + pad)].view(rows, D + pad)[:, :D], flat


def _tokens(kind, N, V, seed=0):
    g = np.random.Generator(np.random.Philox(np.random.SeedSequence([seed, N, V])))
    if kind == "one":
        t = np.full(N, V // 2)
    elif kind == "none":
        t = np.full(N, -100)
    elif kind == "uniform":
        t = g.integers(0, V, N)
    elif kind == "ends":
        t = np.where(g.random(N) < 0.5, 0, V - 1)
    else:   # frequent low ids, some ignored, some out of range
        t = np.floor(V ** g.random(N) - 1).astype(np.int64).clip(0, V - 1)
        t[g.random(N) < 0.1] = -100
        t[g.random(N) < 0.02] = V
        t[g.random(N) < 0.02] = -1
    return torch.from_numpy(t.astype(np.int32)).to(DEV)


def _lookup(W, t, scale):
    y = torch.zeros(t.numel(), W.shape[1], dtype=torch.float64, device=DEV)
    live = (t >= 0) & (t < W.shape[0])
    y[live] = W.double()[t[live].long()] * float(np.float32(scale))
    y[(t != -100) & ~live] = float("nan")
    return y


def _table_grad(dy, t, V, scale):
    """(gradient, sum of magnitudes) in float64."""
    live = (t >= 0) & (t < V)
    zero = torch.zeros(V, dy.shape[1], dtype=torch.float64, device=DEV)
    s = float(np.float32(scale))
    rows = dy.double()[live]
    return (zero.index_add(0, t[live].long(), rows) * s,
            zero.index_add(0, t[live].long(), rows.abs()) * abs(s))


def _grad_bound(N, want, size, old, dtype):
    rng = max(32, -(-(-(-N // 2048)) // 8) * 8) if N else 32
    e = U * (rng + -(-N // rng) / 8 + 12)
    return e * size + 2 * U * (want.abs() + old.abs()) + half_step(dtype) * 1.01 * (want + old).abs() + 2.0 ** -126


@pytest.mark.parametrize("wdtype,dtype", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("N,V,D,pad,shift", [
    (1, 1, 1, 0, 0), (1, 1000, 4096, 0, 0), (3, 7, 3, 0, 0), (40, 100, 64, 0, 0), (33, 500, 100, 0, 0),
    (301, 1000, 1111, 0, 0), (129, 300, 513, 7, 3), (65, 50, 1024, 8, 8), (17, 50, 1024, 4, 4), (1000, 20, 33, 1, 0),
    (5, 9, 20001, 0, 0)])
def test_lookup(wdtype, dtype, N, V, D, pad, shift):
    W, _ = _matrix(V, D, wdtype, N + V, pad, shift)
    t = _tokens("mixed", N, V)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for scale in (1.0, -3.7):
        y = flce.embedding(W, t, scale=scale, dtype=TYPES[dtype])
        want = _lookup(W, t, scale)
        assert y.dtype == TYPES[dtype] and y.shape == (N, D)
        bad = torch.isnan(want)
        assert torch.equal(torch.isnan(y), bad)
        err = (y.double() - want).abs()[~bad]
        # one product in fp32 (none where the scale is 1), one rounding to the type
        assert bool((err <= (half_step(TYPES[dtype]) * 1.01 + U) * want.abs()[~bad]).all())
        out = torch.empty_like(y)
        assert flce.embedding(W, t, scale=scale, out=out, status=status) is out
        assert torch.equal(out.nan_to_num(9.0), y.nan_to_num(9.0))
    has_bad = bool(((t != -100) & ((t < 0) | (t >= V))).any())
    assert flce.check_status(status) == (flce.FLCE_ERR_LABEL_RANGE if has_bad else flce.FLCE_OK)


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("kind,N,V,D,pad,shift", [
    ("mixed", 1, 1, 1, 0, 0), ("mixed", 1, 1000, 4096, 0, 0), ("mixed", 31, 7, 3, 0, 0), ("one", 33, 5, 64, 0, 0),
    ("one", 1024, 40, 256, 0, 0), ("ends", 1025, 70000, 100, 0, 0), ("mixed", 700, 300, 1111, 0, 0),
    ("mixed", 4096, 33, 513, 7, 3), ("none", 200, 100, 96, 0, 0), ("uniform", 5000, 40000, 136, 8, 8),
    ("one", 8193, 3, 40, 4, 4), ("mixed", 16384, 130000, 64, 0, 0), ("uniform", 16385, 300000, 32, 0, 0),
    ("one", 20000, 2, 33, 0, 0), ("mixed", 70000, 1000, 20, 0, 0), ("ends", 140000, 270000, 8, 0, 0),
    ("mixed", 40, 9, 5001, 1, 0)])
def test_table_gradient(dtype, wdtype, kind, N, V, D, pad, shift):
    dy, _ = _matrix(N, D, dtype, N + D, pad, shift)
    t = _tokens(kind, N, V)
    for scale in (1.0, 2.3):
        want, size = _table_grad(dy, t, V, scale)
        got = flce.embedding_backward(dy, t, V, scale=scale, dtype=TYPES[wdtype])
        assert got.dtype == TYPES[wdtype] and got.shape == (V, D)
        zero = torch.zeros_like(want)
        assert bool(((got.double() - want).abs() <= _grad_bound(N, want, size, zero, got.dtype)).all())
        again = flce.embedding_backward(dy, t, V, scale=scale, dtype=TYPES[wdtype])
        assert torch.equal(got, again)
        # into a table in its place among others; and added to one
        out, flat = _matrix(V, D, wdtype, 3, pad, shift)
        before, old = flat.clone(), out.clone().double()
        assert flce.embedding_backward(dy, t, V, scale=scale, out=out) is out and torch.equal(out, got)
        out.copy_(old.to(out.dtype))
        assert torch.equal(flat, before)   # nothing beside the table was written
        flce.embedding_backward(dy, t, V, scale=scale, out=out, accumulate=True)
        assert bool(((out.double() - old - want).abs() <= _grad_bound(N, want, size, old, got.dtype)).all())
        seen = torch.zeros(V, dtype=torch.bool, device=DEV)
        seen[t[(t >= 0) & (t < V)].long()] = True
        assert torch.equal(out[~seen], old[~seen].to(out.dtype))
        out.copy_(old.to(out.dtype))
        assert torch.equal(flat, before)


def test_no_tokens():
    t = torch.zeros(0, dtype=torch.int32, device=DEV)
    W = torch.ones(5, 12, device=DEV)
    assert flce.embedding(W, t).shape == (0, 12)
    dy = torch.zeros(0, 12, device=DEV)
    assert torch.equal(flce.embedding_backward(dy, t, 5), torch.zeros(5, 12, device=DEV))
    assert torch.equal(flce.embedding_backward(dy, t, 5, out=W, accumulate=True), torch.ones(5, 12, device=DEV))


def test_tokens_of_any_shape_and_expanded_gradients():
    W = torch.randn(50, 24, device=DEV)
    t = _tokens("uniform", 30, 50).view(2, 3, 5)
    y = flce.embedding(W, t)
    assert y.shape == (2, 3, 5, 24) and torch.equal(y, W[t.long()])
    one = torch.ones((), device=DEV).expand(2, 3, 5, 24)
    want = torch.bincount(t.flatten().long(), minlength=50).float()[:, None].expand(50, 24)
    assert torch.equal(flce.embedding_backward(one, t, 50), want)


def test_tables_past_2_31_elements():
    V, D = 600_000, 4096
    W = torch.empty(V, D, dtype=torch.bfloat16, device=DEV)
    W.view(V, 64, 64).copy_(torch.arange(64, device=DEV).bfloat16())
    t = torch.tensor([V - 1, 0, 540_000, V - 1], dtype=torch.int32, device=DEV)
    W[t.long()] = torch.randn(4, D, device=DEV).bfloat16()
    y = flce.embedding(W, t)
    assert torch.equal(y, W[t.long()])
    dy = torch.randn(4, D, device=DEV).bfloat16()
    dW = flce.embedding_backward(dy, t, V, out=W)
    assert torch.equal(dW[0], dy[1]) and torch.equal(dW[540_000], dy[2])
    assert torch.equal(dW[V - 1], (dy[0].float() + dy[3].float()).bfloat16())
    for a in range(0, V, 100_000):
        assert int((dW[a:a + 100_000] != 0).any(1).sum()) == sum(a <= k < a + 100_000 for k in (0, 540_000, V - 1))


def test_autograd_against_differences():
    torch.manual_seed(0)
    W = torch.randn(40, 17, device=DEV, requires_grad=True)
    t = _tokens("uniform", 12, 40).long().view(3, 4)
    t[0, 0] = -100
    c = torch.randn(3, 4, 17, device=DEV)
    y = flce.fused_embedding(t, W, scale=1.5)
    (y * c).sum().backward()
    # linear in W: a difference of any step is the derivative, up to fp32 roundings of sums of 17 * 12
    for v, d in ((int(t[0, 1]), 3), (int(t[2, 3]), 16), (0, 0)):
        step = torch.zeros_like(W)
        step[v, d] = 0.5
        with torch.no_grad():
            up = (flce.fused_embedding(t, W + step, scale=1.5).double() * c.double()).sum()
            down = (flce.fused_embedding(t, W - step, scale=1.5).double() * c.double()).sum()
        assert abs(float(up - down) - float(W.grad[v, d])) <= 1e-5 * (1 + abs(float(W.grad[v, d])))
    m = flce.FusedEmbedding(40, 16, scale=4.0, device=DEV, dtype=torch.float32, out_dtype=torch.bfloat16)
    out = m(t)
    assert out.dtype == torch.bfloat16 and bool((out[0, 0] == 0).all())
    out.float().sum().backward()
    count = torch.bincount(t[t >= 0], minlength=40).float()
    assert torch.equal(m.weight.grad, 4.0 * count[:, None].expand(40, 16))


def test_other_streams_and_graphs():
    V, D, N = 900, 264, 3000
    W = torch.randn(V, D, device=DEV).bfloat16()
    dy = torch.randn(N, D, device=DEV).bfloat16()
    t = _tokens("mixed", N, V)
    want_y, want = flce.embedding(W, t).nan_to_num(7.0), flce.embedding_backward(dy, t, V)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, g = flce.embedding(W, t, stream=side), flce.embedding_backward(dy, t, V, stream=side)
    side.synchronize()
    assert torch.equal(y.nan_to_num(7.0), want_y) and torch.equal(g, want)
    t2, dy2 = t.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = flce.embedding(W, t2), flce.embedding_backward(dy2, t2, V)
    for k in range(3):
        t2.copy_(t.roll(k))
        dy2.copy_(dy.roll(k, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.nan_to_num(7.0), want_y.roll(k, 0))
        seen = (flce.embedding_backward(dy2, t2, V))
        assert torch.equal(g, seen)


def test_refusals():
    W = torch.zeros(5, 8, device=DEV)
    t = torch.zeros(3, dtype=torch.int32, device=DEV)
    dy = torch.zeros(3, 8, device=DEV)
    for call, error in (
            (lambda: flce.embedding(W, t.long()), TypeError), (lambda: flce.embedding(W.half(), t), TypeError),
            (lambda: flce.embedding(W.t(), t), ValueError), (lambda: flce.embedding(W, t.cpu()), ValueError),
            (lambda: flce.embedding(W, t, dtype=torch.float16), TypeError),
            (lambda: flce.embedding(W, t, scale=float("inf")), flce.FLCEError),
            (lambda: flce.embedding(W, t, out=torch.zeros(3, 7, device=DEV)), ValueError),
            (lambda: flce.embedding_backward(dy[:2], t, 5), ValueError),
            (lambda: flce.embedding_backward(dy, t, 0), flce.FLCEError),
            (lambda: flce.embedding_backward(dy, t, 5, accumulate=True), ValueError),
            (lambda: flce.embedding_backward(dy, t, 5, out=torch.zeros(4, 8, device=DEV)), ValueError),
            (lambda: flce.embedding_backward(dy, t, 5, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV)),
             flce.FLCEError)):
        with pytest.raises(error):
            call()
