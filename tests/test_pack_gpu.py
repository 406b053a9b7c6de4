"""Activations in 8 bits: codes, scales and values exactly those of the definition; the layer norm
that keeps its input so, against the float64 formulas over the values kept, with the bounds of
test_layer_norm_gpu.py (h = (x~ - mean) rstd has the mean's and rstd's errors and two roundings)."""
import numpy as np
import pytest

from head_ops_testlib import U, half_step
from oracle import block_formats as bf
from oracle import head_ops as ho
from test_layer_norm_gpu import TYPES, _draw, _errors, _put, _within

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"


def _values(N, D, seed):
    """Magnitudes over the whole range, with zeros, ties, tiny and non-finite values among them."""
    g = np.random.Generator(np.random.Philox(np.random.SeedSequence([seed, N, D])))
    x = g.standard_normal((N, D)) * np.exp2(g.integers(-140, 120, (N, 1)) * (g.random((N, 1)) < 0.3))
    x[g.random((N, D)) < 0.05] = 0.0
    tie = g.random((N, D)) < 0.1   # halfway between two codes, whatever the power of two
    x = np.where(tie, np.sign(x) * (2 * g.integers(8, 16, (N, D)) + 1) * np.exp2(g.integers(-8, 3, (N, D))), x)
    x[g.random(N) < 0.05] = 0.0
    x = np.clip(x, -3e38, 3e38)
    x[g.random((N, D)) < 0.2 / D] = np.inf
    x[g.random((N, D)) < 0.2 / D] = np.nan
    x[:, 0] = np.where(g.random(N) < 0.2, -0.0, x[:, 0])
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D,pad,shift", [
    (1, 1, 0, 0), (1, 4096, 0, 0), (3, 31, 0, 0), (5, 32, 0, 0), (2, 33, 3, 1), (40, 64, 0, 0), (33, 100, 4, 0),
    (20, 136, 0, 0), (9, 513, 7, 3), (7, 1111, 0, 0), (64, 520, 8, 8), (2, 8200, 0, 0), (200, 24, 0, 0),
    (3, 5001, 0, 1)])
def test_codes_scales_and_values(dtype, N, D, pad, shift):
    xt, x = _put(_values(N, D, 7), dtype, pad, shift)
    p = flce.pack_e4m3(xt)
    codes, scales, values = bf.pack_e4m3(x)
    assert np.array_equal(p.scales.cpu().numpy(), scales)
    assert np.array_equal(p.codes.cpu().numpy(), codes)
    rest = p.data.clone()   # what lies behind the codes and behind the scales is 0
    blocks = -(-D // 32)
    rest[:, :D] = 0
    rest[:, 32 * blocks:33 * blocks] = 0
    assert not bool(rest.any())
    got = flce.unpack_e4m3(p, dtype=torch.float32).cpu().numpy()
    assert np.array_equal(got, values.astype(np.float32), equal_nan=True)
    want = torch.from_numpy(values.astype(np.float32)).bfloat16()
    got = flce.unpack_e4m3(p, dtype=torch.bfloat16).cpu()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(1.0), want.nan_to_num(1.0))
    out = torch.empty_like(got, device=DEV)
    assert flce.unpack_e4m3(p, out=out, dtype=torch.bfloat16) is out


def test_any_shape_and_outputs_in_place_among_others():
    x = torch.randn(2, 3, 5, 72, device=DEV).bfloat16()
    p = flce.pack_e4m3(x)
    assert p.shape == (2, 3, 5, 72) and p.data.shape == (30, flce.packed_row_bytes(72))
    y = flce.unpack_e4m3(p)
    assert y.shape == x.shape and y.dtype == x.dtype
    assert bool(((y - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -9).all())
    buf = torch.full((32, flce.packed_row_bytes(72)), 9, dtype=torch.uint8, device=DEV)
    q = flce.pack_e4m3(x, out=buf[1:31])
    assert torch.equal(q.data, p.data) and bool((buf[0] == 9).all()) and bool((buf[31] == 9).all())
    view = x.transpose(0, 1)
    assert torch.equal(flce.unpack_e4m3(flce.pack_e4m3(view)), y.transpose(0, 1))
    none = flce.pack_e4m3(torch.zeros(0, 8, device=DEV))
    assert flce.unpack_e4m3(none).shape == (0, 8)


def _run(x, dy, w, b, dtype, wdtype, *, pad=0, shift=0, gpad=None, gshift=None):
    xt, x = _put(x, dtype, pad, shift)
    wt, w = _put(w, wdtype) if w is not None else (None, None)
    bt, b = _put(b, wdtype) if b is not None else (None, None)
    r, packed = flce.layer_norm_packed(xt, wt, bt)
    y, mean, rstd = ho.layer_norm(x, w, b, 1e-5)
    e, h, dh = _errors(x, mean, rstd)
    aw, ab = (1.0 if w is None else np.abs(w)), (0.0 if b is None else np.abs(b))
    _within(r.mean, mean, e * np.abs(x).mean(axis=1) + U * np.abs(mean), "mean")
    _within(r.rstd, rstd, rstd * (2 * e + 8 * U + (e * np.abs(x).mean(axis=1) * rstd) ** 2), "rstd")
    _within(r.y, y, aw * dh + 2 * U * (np.abs(h) * aw + ab) + half_step(r.y.dtype) * np.abs(y) * 1.01, "y")
    assert torch.equal(packed.data, flce.pack_e4m3(xt).data)
    kept = flce.unpack_e4m3(packed, dtype=torch.float32).double().cpu().numpy()
    dyt, dy = _put(dy, dtype, pad if gpad is None else gpad, shift if gshift is None else gshift)
    got = flce.layer_norm_packed_backward(dyt, packed, wt, r)
    D = x.shape[1]
    h = (kept - mean[:, None]) * rstd[:, None]
    dm = e * np.abs(x).mean(axis=1)
    dh = (2 * e + 8 * U) * np.abs(h) + (dm * rstd)[:, None] + np.abs(h) * ((dm * rstd) ** 2)[:, None]
    g = dy * (1.0 if w is None else w)
    ag = np.abs(g)
    mg, mgh = g.mean(axis=1, keepdims=True), (g * h).mean(axis=1, keepdims=True)
    rx = rstd[:, None] * (g - mg - h * mgh)
    err_mg = (e + U) * ag.mean(axis=1, keepdims=True)
    err_mgh = (e + U) * (ag * np.abs(h)).mean(axis=1, keepdims=True) + (ag * dh).mean(axis=1, keepdims=True)
    size = ag + np.abs(mg) + np.abs(h) * np.abs(mgh)
    bound = rstd[:, None] * (err_mg + np.abs(h) * err_mgh + dh * np.abs(mgh) + (2 * e + 10 * U) * size)
    _within(got[0], rx, bound + half_step(got[0].dtype) * np.abs(rx) * 1.01, "dx")
    en = U * (x.shape[0] / 16 + 400)
    rw, rb = (dy * h).sum(axis=0), dy.sum(axis=0)
    _within(got[1], rw, (np.abs(dy) * (dh + en * np.abs(h))).sum(axis=0) + half_step(got[1].dtype) * np.abs(rw) * 1.01, "dw")
    _within(got[2], rb, en * np.abs(dy).sum(axis=0) + half_step(got[2].dtype) * np.abs(rb) * 1.01, "db")
    assert D == got[1].numel()
    return dyt, packed, wt, r, got


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("N,D,pad,shift", [
    (1, 1, 0, 0), (3, 2, 0, 0), (2, 100, 0, 0), (7, 127, 0, 0), (1, 4096, 0, 0), (33, 520, 0, 0), (301, 1111, 0, 0),
    (700, 2048, 0, 0), (9, 4095, 0, 0), (3, 8192, 0, 0), (2, 16384, 0, 0), (2, 20001, 0, 0), (3000, 96, 0, 0),
    (6, 513, 7, 3), (20, 2048, 64, 8), (2001, 512, 0, 0), (1501, 1032, 24, 0), (701, 4096, 0, 0), (305, 8192, 0, 0),
    (2000, 511, 0, 0), (1501, 1030, 0, 1), (1203, 2731, 5, 0), (303, 8190, 2, 0), (900, 4095, 0, 3)])
def test_layer_norm(dtype, wdtype, N, D, pad, shift):
    x, dy, w, b = _draw(N, D, N + D)
    _run(x, dy, w, b, dtype, wdtype, pad=pad, shift=shift)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,pad,shift,gpad,gshift", [(2501, 1000, 3, 1, 0, 0), (2501, 1024, 0, 0, 5, 2),
                                                       (1501, 1111, 1, 0, 0, 2), (40, 264, 0, 0, 3, 1)])
def test_layer_norm_in_parts_in_place_and_in_other_strides(dtype, N, D, pad, shift, gpad, gshift):
    x, dy, w, b = _draw(N, D, D)
    dyt, packed, wt, r, want = _run(x, dy, w, b, dtype, "f32", pad=pad, shift=shift, gpad=gpad, gshift=gshift)
    _run(x, dy, None, b, dtype, "f32", pad=pad, shift=shift, gpad=gpad, gshift=gshift)
    for k in range(3):
        need = [i == k for i in range(3)]
        got = flce.layer_norm_packed_backward(dyt, packed, wt, r, need_dx=need[0], need_dweight=need[1], need_dbias=need[2])
        assert [g is None for g in got] == [i != k for i in range(3)]
        # (a dense gradient without dx may go by another kernel than one in other strides)
        if gpad == 0 or k == 0:
            assert torch.equal(got[k], want[k])
    # dx into dy; y into x
    dense = dyt.contiguous()
    first = flce.layer_norm_packed_backward(dense, packed, wt, r)
    assert torch.equal(flce.layer_norm_packed_backward(dense, packed, wt, r, out={"dx": dense})[0], first[0])
    xt = _put(x, dtype)[0]
    want_y, want_p = flce.layer_norm_packed(xt, wt)
    buf = torch.empty_like(want_p.data)
    got_y, got_p = flce.layer_norm_packed(xt, wt, out={"y": xt, "packed": buf})
    assert got_y.y is xt and torch.equal(xt, want_y.y) and got_p.data is buf and torch.equal(buf, want_p.data)


@pytest.mark.parametrize("N,D,wdtype", [(16395, 1032, "f32"), (2051, 8200, "bf16")])
def test_layer_norm_of_many_bf16_rows(N, D, wdtype):
    x, dy, w, b = _draw(N, D, N + D)
    _run(x, dy, w, b, "bf16", wdtype)
    xt = _put(_values(N, D, 11), "bf16")[0]
    r, packed = flce.layer_norm_packed(xt)
    assert torch.equal(packed.data, flce.pack_e4m3(xt).data)
    bad = ~xt.isfinite().all(dim=1)
    assert bool(bad.any()) and bool(r.y[bad].isnan().any(dim=1).all()) and bool(r.mean[~bad].isfinite().all())


def test_no_rows():
    x = torch.zeros(0, 40, device=DEV)
    r, p = flce.layer_norm_packed(x)
    dx, dw, db = flce.layer_norm_packed_backward(x, p, None, r)
    assert dx.shape == (0, 40) and not bool(dw.any()) and not bool(db.any())


def test_autograd_keeps_8_bits():
    torch.manual_seed(1)
    x = torch.randn(6, 50, 96, device=DEV).bfloat16().requires_grad_()
    n = flce.FusedLayerNorm(96, device=DEV, packed=True)
    with torch.no_grad():
        n.weight.normal_(1, 0.1)
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (kept.append(t.numel() * t.element_size()), t)[1], lambda t: t):
        y = n(x)
    assert max(kept) == 300 * flce.packed_row_bytes(96)
    c = torch.randn_like(y)
    (y * c).sum().backward()
    r, p = flce.layer_norm_packed(x.detach(), n.weight.detach(), n.bias.detach())
    dx, dw, db = flce.layer_norm_packed_backward(c, p, n.weight.detach(), r)
    assert torch.equal(x.grad, dx) and torch.equal(n.weight.grad, dw) and torch.equal(n.bias.grad, db)
    # near the gradients from x itself: h is off by 2^-4 at most of x, dx and dweight by as much of their terms
    x2 = x.detach().requires_grad_()
    m = flce.FusedLayerNorm(96, device=DEV)
    m.load_state_dict(n.state_dict())
    (m(x2) * c).sum().backward()
    assert float((x.grad - x2.grad).double().norm() / x2.grad.double().norm()) <= 2.0 ** -4
    assert torch.equal(n.bias.grad, m.bias.grad)


def test_graphs_and_streams():
    x = torch.randn(3000, 1024, device=DEV).bfloat16()
    dy = torch.randn_like(x)
    w = torch.randn(1024, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r, p = flce.layer_norm_packed(x, w, stream=side)
    got = flce.layer_norm_packed_backward(dy, p, w, r, stream=side)
    v = flce.unpack_e4m3(flce.pack_e4m3(x, stream=side), stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r2, p2 = flce.layer_norm_packed(x, w)
        again = flce.layer_norm_packed_backward(dy, p2, w, r2)
        v2 = flce.unpack_e4m3(p2)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(v, v2) and torch.equal(r.y, r2.y) and all(torch.equal(a, b) for a, b in zip(got, again))


def test_refusals():
    x = torch.zeros(3, 40, device=DEV)
    r, p = flce.layer_norm_packed(x)
    short = flce.PackedRows(p.data[:2], p.shape, p.dtype)
    for call, error in (
            (lambda: flce.pack_e4m3(x.half()), TypeError), (lambda: flce.pack_e4m3(x.cpu()), ValueError),
            (lambda: flce.pack_e4m3(x, out=torch.zeros(3, 40, dtype=torch.uint8, device=DEV)), ValueError),
            (lambda: flce.unpack_e4m3(p, dtype=torch.float16), TypeError), (lambda: flce.unpack_e4m3(short), ValueError),
            (lambda: flce.unpack_e4m3(p, out=torch.zeros(3, 41, device=DEV)), ValueError),
            (lambda: flce.layer_norm_packed(x, eps=-1.0), flce.FLCEError),
            (lambda: flce.layer_norm_packed(x, torch.ones(41, device=DEV)), ValueError),
            (lambda: flce.layer_norm_packed_backward(x.bfloat16(), p, None, r), ValueError),
            (lambda: flce.layer_norm_packed_backward(x[:2], p, None, r), ValueError),
            (lambda: flce.layer_norm_packed_backward(x, short, None, r), ValueError)):
        with pytest.raises(error):
            call()
