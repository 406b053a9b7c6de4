"""Layer norm and its gradients against the float64 definitions.

Bounds, u = 2^-24: a mean over D values is off by e mean|x|, e = u (D / 64 + 24) (a chain of
at most D / 64 additions, then trees); the variance, from centred values, by 2 e of itself and
the square of the mean's error; so h = (x - mean) rstd by dh = (2 e + 8 u) |h| + e mean|x| rstd.
Sums over N rows add u (N / 16 + 400). Each output is rounded once to its type."""
import numpy as np
import pytest

from head_ops_testlib import U, half_step
from oracle import head_ops as ho

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _rng(seed):
    return np.random.Generator(np.random.Philox(np.random.SeedSequence([seed, 63])))


def _put(x, dtype, pad=0, shift=0):
    """Rounded to dtype on the device, with row stride D + pad and an element offset, and
    the float64 values it holds."""
    x = np.asarray(x, dtype=np.float32)
    if x.ndim == 1:
        t = torch.from_numpy(x).to(DEV).to(TYPES[dtype])
        return t, t.double().cpu().numpy()
    N, D = x.shape
    flat = torch.zeros(shift + N * (D + pad), dtype=TYPES[dtype], device=DEV)
    t = flat[shift:].view(N, D + pad)[:, :D]
    t.copy_(torch.from_numpy(x))
    return t, t.double().cpu().numpy()


def _errors(x, mean, rstd):
    D = x.shape[1]
    e = U * (D / 64 + 24)
    h = (x - mean[:, None]) * rstd[:, None]
    dm = e * np.abs(x).mean(axis=1)
    return e, h, (2 * e + 8 * U) * np.abs(h) + (dm * rstd)[:, None] + np.abs(h) * ((dm * rstd) ** 2)[:, None]


def _within(got, want, bound, name):
    got = got.double().cpu().numpy()
    err = np.abs(got - want)
    assert np.all(err <= bound), (name, float(np.max(err / np.maximum(bound, 1e-300))))


def _run(x, dy, w, b, dtype, wdtype, *, eps=1e-5, pad=0, shift=0):
    xt, x = _put(x, dtype, pad, shift)
    wt, w = _put(w, wdtype) if w is not None else (None, None)
    bt, b = _put(b, wdtype) if b is not None else (None, None)
    r = flce.layer_norm(xt, wt, bt, eps=eps)
    assert r.y.dtype == xt.dtype
    y, mean, rstd = ho.layer_norm(x, w, b, eps)
    e, h, dh = _errors(x, mean, rstd)
    aw = 1.0 if w is None else np.abs(w)
    ab = 0.0 if b is None else np.abs(b)
    _within(r.mean, mean, e * np.abs(x).mean(axis=1) + U * np.abs(mean), "mean")
    _within(r.rstd, rstd, rstd * (2 * e + 8 * U + (e * np.abs(x).mean(axis=1) * rstd) ** 2), "rstd")
    _within(r.y, y, aw * dh + 2 * U * (np.abs(h) * aw + ab) + half_step(r.y.dtype) * np.abs(y) * 1.01, "y")
    if dy is None:
        return
    dyt, dy = _put(dy, dtype, pad, shift)
    dx, dw, db = flce.layer_norm_backward(dyt, xt, wt, r)
    rx, rw, rb = ho.layer_norm_grad(dy, x, w, eps)
    g = dy * (1.0 if w is None else w)
    ag = np.abs(g)
    err_mg = (e + U) * ag.mean(axis=1, keepdims=True)
    err_mgh = (e + U) * (ag * np.abs(h)).mean(axis=1, keepdims=True) + (ag * dh).mean(axis=1, keepdims=True)
    mgh = np.abs((g * h).mean(axis=1, keepdims=True))
    size = ag + np.abs(g.mean(axis=1, keepdims=True)) + np.abs(h) * mgh
    bound = rstd[:, None] * (err_mg + np.abs(h) * err_mgh + dh * mgh + (2 * e + 10 * U) * size)
    _within(dx, rx, bound + half_step(dx.dtype) * np.abs(rx) * 1.01, "dx")
    en = U * (x.shape[0] / 16 + 400)
    _within(dw, rw, (np.abs(dy) * (dh + en * np.abs(h))).sum(axis=0) + half_step(dw.dtype) * np.abs(rw) * 1.01, "dw")
    _within(db, rb, en * np.abs(dy).sum(axis=0) + half_step(db.dtype) * np.abs(rb) * 1.01, "db")


def _draw(N, D, seed):
    g = _rng(seed)
    x = g.standard_normal((N, D)) * (1 + 7 * (g.random(D) < 0.02)) + 0.25
    return x, g.standard_normal((N, D)) * 1e-2, 1 + 0.1 * g.standard_normal(D), 0.1 * g.standard_normal(D)


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("N,D", [
    (1, 1), (3, 2), (1, 64), (2, 100), (7, 127), (40, 128), (1, 4096), (33, 520), (301, 1111),
    (5, 1024), (700, 2048), (9, 4095), (4, 5120), (3, 8192), (2, 8200), (2, 16384), (2, 20001),
    (1, 40000), (3000, 96), (5000, 33)])
def test_shapes_and_types(dtype, wdtype, N, D):
    x, dy, w, b = _draw(N, D, N + D)
    _run(x, dy, w, b, dtype, wdtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,pad,shift", [(5, 256, 8, 0), (5, 256, 3, 0), (4, 1000, 0, 1), (6, 513, 7, 3),
                                           (3, 4096, 1, 0), (20, 2048, 64, 8)])
def test_strides_and_alignments(dtype, N, D, pad, shift):
    x, dy, w, b = _draw(N, D, N + D + pad)
    _run(x, dy, w, b, dtype, "f32", pad=pad, shift=shift)


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("N,D,pad", [
    (2001, 512, 0), (4000, 512, 24), (1501, 1032, 0), (1203, 2728, 8), (701, 4096, 0), (305, 8192, 0),
    (153, 12288, 0), (160, 16384, 8), (2000, 511, 0), (1501, 1030, 0), (1203, 2731, 5), (701, 4095, 0),
    (303, 8190, 2)])
def test_many_rows(dtype, wdtype, N, D, pad):
    x, dy, w, b = _draw(N, D, N + D)
    _run(x, dy, w, b, dtype, wdtype, pad=pad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,pad,shift", [(1024, 0, 0), (1000, 3, 1), (1029, 0, 2), (1111, 5, 0), (1031, 8, 3)])
def test_many_rows_in_place_and_in_parts(dtype, D, pad, shift):
    N = 2501
    x, dy, w, b = _draw(N, D, D)
    xt, dyt = (_put(a, dtype, pad, shift)[0] for a in (x, dy))
    wt, bt = (_put(a, "f32")[0] for a in (w, b))
    r = flce.layer_norm(xt, wt, bt)
    want = flce.layer_norm_backward(dyt, xt, wt, r)
    for k in range(3):
        need = [i == k for i in range(3)]
        got = flce.layer_norm_backward(dyt, xt, wt, r, need_dx=need[0], need_dweight=need[1], need_dbias=need[2])
        assert torch.equal(got[k], want[k])
    if pad == 0:   # outputs are contiguous
        g = _put(dy, dtype, pad, shift)[0]
        assert torch.equal(flce.layer_norm_backward(g, xt, wt, r, out={"dx": g})[0], want[0])
        y = _put(x, dtype, pad, shift)[0]
        assert torch.equal(flce.layer_norm(y, wt, bt, out={"y": y}).y, r.y)
    for got in (flce.layer_norm(xt, wt).y, flce.layer_norm(xt, None, bt).y, flce.layer_norm(xt).y):
        assert got.shape == (N, D) and bool(torch.isfinite(got).all())
    _run(x, dy, w, None, dtype, "f32", pad=pad, shift=shift)
    _run(x, dy, None, b, dtype, "bf16", pad=pad, shift=shift)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,xpad,gpad", [(1000, 3, 0), (1024, 0, 5), (1111, 1, 0), (2048, 8, 16)])
def test_rows_and_upstream_gradients_in_different_strides(dtype, D, xpad, gpad):
    N = 1501
    x, dy, w, b = _draw(N, D, D + xpad)
    wt = _put(w, "f32")[0]
    same = _put(x, dtype)[0], _put(dy, dtype)[0]
    want = flce.layer_norm_backward(same[1], same[0], wt, flce.layer_norm(same[0], wt))
    xt, gt = _put(x, dtype, xpad)[0], _put(dy, dtype, gpad)[0]
    r = flce.layer_norm(xt, wt)
    assert r.y.is_contiguous()
    got = flce.layer_norm_backward(gt, xt, wt, r)
    # the same values in another order of sums: by twice their bound of test_shapes_and_types
    e = U * (D / 64 + 24)
    scale = [float(t.double().abs().max()) for t in want]
    n = U * (N / 16 + 400)
    for k, (g, t) in enumerate(zip(got, want)):
        bound = 2 * (8 * e if k == 0 else n * float(np.abs(dy).sum(0).max()) * 8 / max(scale[k], 1e-30)) * scale[k]
        bound += 2 * half_step(t.dtype) * scale[k]
        assert float((g.double() - t.double()).abs().max()) <= bound, k


@pytest.mark.parametrize("with_w,with_b", [(True, False), (False, True), (False, False)])
def test_without_weight_or_bias(with_w, with_b):
    x, dy, w, b = _draw(50, 320, 3)
    _run(x, dy, w if with_w else None, b if with_b else None, "f32", "f32")


def test_constant_rows_and_a_large_mean():
    x, dy, w, b = _draw(6, 512, 4)
    x[0] = 0.0
    x[1] = 3.0
    x[2] += 1000.0
    x[3] *= 1e-6
    x[4] = x[4] * 1e4
    _run(x, dy, w, b, "f32", "f32")
    _run(x, dy, w, b, "f32", "f32", eps=1e-2)


def test_nan_stays_in_its_row():
    x, dy, w, b = _draw(5, 300, 5)
    x[2, 7] = np.nan
    x[3, 0] = np.inf
    xt, _ = _put(x, "f32")
    r = flce.layer_norm(xt, *(_put(t, "f32")[0] for t in (w, b)))
    bad = torch.tensor([False, False, True, True, False], device=DEV)
    assert torch.equal(torch.isnan(r.y).any(1), bad)
    dx, _, _ = flce.layer_norm_backward(_put(dy, "f32")[0], xt, None, r, need_dweight=False, need_dbias=False)
    assert torch.equal(torch.isnan(dx).any(1), bad)


def test_in_place_selected_gradients_and_shapes():
    x, dy, w, b = _draw(24, 640, 6)
    xt, wt, bt, dyt = (_put(t, "bf16")[0] for t in (x, w, b, dy))
    r = flce.layer_norm(xt.view(2, 12, 640), wt, bt)
    assert r.y.shape == (2, 12, 640) and r.mean.shape == (24,)
    want = flce.layer_norm_backward(dyt, xt, wt, r)
    for k in range(3):
        need = [i == k for i in range(3)]
        got = flce.layer_norm_backward(dyt, xt, wt, r, need_dx=need[0], need_dweight=need[1], need_dbias=need[2])
        for i in range(3):
            assert got[i] is None if not need[i] else torch.equal(got[i], want[i])
    g = dyt.clone()
    dx, dw, db = flce.layer_norm_backward(g, xt, wt, r, out={"dx": g})
    assert dx is g and torch.equal(g, want[0]) and torch.equal(dw, want[1]) and torch.equal(db, want[2])
    y = xt.clone()
    assert flce.layer_norm(y, wt, bt, out={"y": y}).y is y and torch.equal(y, r.y.view(24, 640))


def test_no_rows():
    x = torch.empty(0, 16, device=DEV)
    w = torch.ones(16, device=DEV)
    r = flce.layer_norm(x, w)
    dx, dw, db = flce.layer_norm_backward(x, x, w, r)
    assert dx.shape == (0, 16) and torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0


def test_row_offsets_past_32_bits():
    N, D = 600000, 4096
    x = torch.zeros(N, D, dtype=torch.bfloat16, device=DEV)
    x[N - 1].copy_(torch.from_numpy(_draw(1, D, 8)[0][0].astype(np.float32)))
    dy = torch.zeros_like(x)
    dy[N - 1] = 1.0
    dy[N - 1, ::2] = -0.5
    r = flce.layer_norm(x, out=None)
    y, mean, rstd = ho.layer_norm(x[N - 1:].double().cpu().numpy(), None, None, 1e-5)
    assert np.max(np.abs(r.y[N - 1].double().cpu().numpy() - y[0])) <= 2.0 ** -8 * np.max(np.abs(y)) + 1e-5
    dx, dw, db = flce.layer_norm_backward(dy, x, None, r, out={"dx": dy})
    assert float(db[0]) == -0.5 and float(db[1]) == 1.0
    assert torch.count_nonzero(dx[:N - 1]) == 0 and torch.count_nonzero(dx[N - 1]) > 0


def test_repeats_streams_graphs_and_autograd():
    x, dy, w, b = _draw(500, 1024, 9)
    xt, wt, bt, dyt = (_put(t, "bf16")[0] for t in (x, w, b, dy))
    r = flce.layer_norm(xt, wt, bt)
    want = flce.layer_norm_backward(dyt, xt, wt, r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r2 = flce.layer_norm(xt, wt, bt, stream=side)
    got = flce.layer_norm_backward(dyt, xt, wt, r2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(r.y, r2.y) and all(torch.equal(p, q) for p, q in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r2 = flce.layer_norm(xt, wt, bt)
        got = flce.layer_norm_backward(dyt, xt, wt, r2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    m = flce.FusedLayerNorm(1024, device=DEV, dtype=torch.bfloat16)
    with torch.no_grad():
        m.weight.copy_(wt)
        m.bias.copy_(bt)
    leaf = xt.detach().clone().requires_grad_(True)
    m(leaf).sum().backward()      # an expanded upstream gradient
    ones = torch.ones_like(xt)
    want = flce.layer_norm_backward(ones, xt, wt, r)
    assert torch.equal(leaf.grad, want[0]) and torch.equal(m.weight.grad, want[1]) and torch.equal(m.bias.grad, want[2])
