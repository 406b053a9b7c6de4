"""The global gradient norm and clipping against float64. Bounds, u = 2^-24: squares and their
sums of at most 32 terms in fp32 make the sum of squares off by 34 u of itself, the norm by
half of that and its own rounding; the factor adds three roundings and each product one, then
the rounding to the output's type."""
import numpy as np
import pytest

from head_ops_testlib import U, half_step
from oracle import head_ops as ho

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"
NORM_TOL = 20 * U


def _grads(shapes, types, seed, std=3e-3, shift=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    out = []
    for sh, t in zip(shapes, types):
        n = int(np.prod(sh))
        flat = torch.empty(n + shift, dtype=t, device=DEV)
        flat.copy_(torch.randn(n + shift, generator=g, device=DEV) * std)
        out.append(flat[shift:].view(sh))
    return out


def _check(grads, max_norm, out_shift=None):
    host = [g.double().cpu().numpy() for g in grads]
    norm = ho.grad_norm(host)
    c = ho.clip_coefficient(norm, max_norm)
    n = flce.grad_norm(grads)
    assert n.dtype == torch.float32 and n.shape == (1,)
    assert abs(float(n) - norm) <= NORM_TOL * norm
    outs = None
    if out_shift is not None:
        outs = [torch.full((g.numel() + out_shift,), 9.0, dtype=g.dtype, device=DEV)[out_shift:].view(g.shape)
                for g in grads]
    n2 = flce.clip_grads(grads, max_norm, out=outs)
    assert torch.equal(n, n2)
    for g, h, o in zip(grads, host, outs or grads):
        want = h * c
        bound = (half_step(g.dtype) * 1.01 + NORM_TOL + 5 * U) * np.abs(want) + 2.0 ** -149
        if c == 1.0:
            bound = np.zeros_like(want)
        assert np.all(np.abs(o.double().cpu().numpy() - want) <= bound)
        if outs is not None:
            assert np.array_equal(g.double().cpu().numpy(), h)   # the gradients are kept


F, H = torch.float32, torch.bfloat16


@pytest.mark.parametrize("max_norm", [0.1, 1e9, 0.0])
@pytest.mark.parametrize("shapes,types", [
    ([(1,)], [F]), ([(1,)], [H]), ([(7, 3)], [H]), ([(1000, 64), (64,), (3, 5, 7)], [H, F, H]),
    ([(8192,), (8193,), (16384,), (16385,)], [F, H, F, H]), ([(1000003,)], [H]),
    ([(17,)] * 300, [F, H, H] * 100), ([(0,), (5,), (0, 4)], [F, F, H])])
def test_norm_and_clip(shapes, types, max_norm):
    _check(_grads(shapes, types, len(shapes)), max_norm)
    _check(_grads(shapes, types, len(shapes) + 1), max_norm, out_shift=0)


@pytest.mark.parametrize("shift,out_shift", [(1, 1), (3, 0), (0, 5), (7, 2)])
def test_alignments(shift, out_shift):
    for types in ([F, H, F], [H, H, H]):
        _check(_grads([(100003,), (9, 11), (33000,)], types, 5, shift=shift), 0.05, out_shift=out_shift)
        _check(_grads([(100003,), (9, 11), (33000,)], types, 6, shift=shift), 0.05)


def test_no_gradients_and_zero_gradients():
    assert float(flce.grad_norm([])) == 0.0
    assert float(flce.clip_grads([], 1.0)) == 0.0
    z = torch.zeros(1000, device=DEV)
    assert float(flce.clip_grads([z], 0.0)) == 0.0 and torch.count_nonzero(z) == 0


def test_more_tensors_than_one_table_and_a_large_one():
    _check(_grads([(i % 50 + 1, 3) for i in range(500)], [F, H] * 250, 7), 0.02)
    big = torch.full((3_000_000_000,), 2.0 ** -10, dtype=H, device=DEV)   # past 2^31 elements
    small = torch.full((5,), 4.0, device=DEV)
    n = float(flce.clip_grads([small, big], 1.0))
    want = np.sqrt(3e9 * 2.0 ** -20 + 80.0)
    assert abs(n - want) <= NORM_TOL * want
    assert float(big[-1]) == float(big[0]) == float(torch.tensor(2.0 ** -10 / (n + 1e-6)).to(H))
    assert abs(float(small[0]) * (n + 1e-6) / 4.0 - 1) < 8 * U


def test_values_that_are_not_finite():
    for bad in (np.inf, -np.inf, np.nan):
        a, b = _grads([(100,), (50,)], [F, H], 8)
        a[3] = bad
        n = float(flce.clip_grads([a, b], 1.0))
        if np.isnan(bad):
            assert np.isnan(n) and torch.isnan(a).all() and torch.isnan(b).all()
        else:
            assert n == np.inf and torch.isnan(a).sum() == 1 and torch.count_nonzero(b) == 0


def test_dense_orders_and_refusals():
    a, = _grads([(40, 30)], [F], 9)
    t = a.clone().t()
    host = t.cpu().double().numpy()
    n = float(flce.clip_grads([t], 0.01))
    want = host * ho.clip_coefficient(ho.grad_norm([host]), 0.01)
    assert np.allclose(t.cpu().double().numpy(), want, rtol=1e-5, atol=0) and n > 0.01
    with pytest.raises(ValueError):
        flce.clip_grads([a[:, :7]], 1.0)
    with pytest.raises(ValueError):
        flce.clip_grads([a[:1].expand(5, 30)], 1.0)
    with pytest.raises(TypeError):
        flce.grad_norm([a.half()])
    with pytest.raises(ValueError):
        flce.clip_grads([a], 1.0, out=[a[:2]])
    with pytest.raises(flce.FLCEError):
        flce.clip_grads([a], -1.0)


def test_repeats_streams_and_graphs():
    grads = _grads([(3000, 700), (700,), (123457,)], [H, F, H], 10)
    outs = [torch.empty_like(g) for g in grads]
    want_n = flce.clip_grads(grads, 0.1, out=outs)
    want = [o.clone() for o in outs]
    for _ in range(5):
        assert torch.equal(flce.clip_grads(grads, 0.1, out=outs), want_n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n = flce.clip_grads(grads, 0.1, out=outs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(n, want_n) and all(torch.equal(a, b) for a, b in zip(outs, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = flce.clip_grads(grads, 0.1)
    copies = [g.clone() for g in grads]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(n, want_n) and all(torch.equal(a, b) for a, b in zip(grads, want))
    graph.replay()      # reads the gradients afresh: now of norm 0.1
    torch.cuda.synchronize()
    assert abs(float(n) - 0.1) < 1e-3 and not torch.equal(grads[0], copies[0])
