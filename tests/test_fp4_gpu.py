"""4-bit floating point: codes, scales and values exactly those of the definition; products against
float64 over the values.

Bound of a product, S = |H~| |W~|^T: codes and scales multiply exactly; a step of 64 values is aligned
to its largest term and added to the sum, each time off by at most 2^-22 of the magnitudes so far
(twice a truncation to 24 bits), so (D / 64 + 4) 2^-22 S, two roundings of the rows' scales and the
type's one."""
import numpy as np
import pytest

from head_ops_testlib import U, half_step
from oracle import block_formats as bf
from test_layer_norm_gpu import _put
from test_pack_gpu import _values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _row_codes(m):
    """The codes one to a byte, [rows, padded width]."""
    c = m.codes.cpu().numpy()
    return np.stack([c & 15, c >> 4], axis=2).reshape(c.shape[0], -1)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D,pad,shift", [
    (1, 1, 0, 0), (1, 4096, 0, 0), (3, 31, 0, 0), (5, 32, 0, 0), (2, 33, 3, 1), (40, 64, 0, 0), (33, 100, 4, 0),
    (129, 136, 0, 0), (9, 513, 7, 3), (260, 72, 0, 0), (7, 1111, 0, 0), (64, 520, 8, 8), (2, 8200, 0, 0),
    (1, 40000, 0, 0), (700, 24, 0, 0)])
def test_codes_scales_and_values(fmt, dtype, N, D, pad, shift):
    xt, x = _put(_values(N, D, 9), dtype, pad, shift)
    m = flce.quantize_fp4(xt, format=fmt)
    codes, scales, rows, values = bf.quantize_fp4(x, fmt)
    if fmt == "nvfp4":
        assert np.array_equal(m.row_scales.cpu().numpy(), rows)
    else:
        assert m.row_scales is None
    assert np.array_equal(m.block_scales().cpu().numpy(), scales)
    got = _row_codes(m)
    assert np.array_equal(got[:, :D], codes) and not got[:, D:].any()
    again = flce.Fp4Matrix.from_rows(m.codes[:, :(D + 1) // 2], m.block_scales(), m.row_scales, width=D, format=fmt)
    assert torch.equal(again.scales, m.scales) and torch.equal(again.codes, m.codes)   # padding too
    got = flce.dequantize_fp4(m).cpu().numpy()
    assert np.array_equal(got, values.astype(np.float32), equal_nan=True)
    want = torch.from_numpy(values.astype(np.float32)).bfloat16()
    got = flce.dequantize_fp4(m, dtype=torch.bfloat16).cpu()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(1.0), want.nan_to_num(1.0))


def test_any_shape_and_row_scales():
    x = torch.randn(2, 3, 72, device=DEV).bfloat16()
    m = flce.quantize_fp4(x)
    assert m.shape == (2, 3, 72) and flce.dequantize_fp4(m).shape == (2, 3, 72)
    view = x.transpose(0, 1)
    assert torch.equal(flce.dequantize_fp4(flce.quantize_fp4(view)), flce.dequantize_fp4(m).transpose(0, 1))
    g = torch.rand(6, device=DEV) + 0.5   # any row scales, as a checkpoint may have them
    n = flce.Fp4Matrix.from_rows(m.codes[:, :36], m.block_scales(), g, width=72)
    plain = flce.Fp4Matrix.from_rows(m.codes[:, :36], m.block_scales(), width=72)
    assert torch.equal(flce.dequantize_fp4(n), flce.dequantize_fp4(plain) * g[:, None])
    for fmt in flce.FP4_FORMATS:
        none = flce.quantize_fp4(torch.zeros(0, 40, device=DEV), format=fmt)
        assert flce.dequantize_fp4(none).shape == (0, 40)
        assert flce.linear_fp4(none, flce.quantize_fp4(x[0, :, :40].contiguous(), format=fmt)).shape == (0, 3)


def _pair(N, D, V, fmt, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(N, D, generator=g, device=DEV) * torch.exp(torch.randn(N, 1, generator=g, device=DEV))
    w = torch.randn(V, D, generator=g, device=DEV) * torch.exp(torch.randn(V, 1, generator=g, device=DEV))
    return flce.quantize_fp4(x.bfloat16(), format=fmt), flce.quantize_fp4(w, format=fmt)


def _check(y, h, w):
    a, b = flce.dequantize_fp4(h).double(), flce.dequantize_fp4(w).double()
    want, size = a @ b.T, a.abs() @ b.abs().T
    D = a.shape[1]
    bound = (-(-D // 64) + 4) * 2.0 ** -22 * size + 2 * U * want.abs() + half_step(y.dtype) * 1.01 * want.abs()
    err = (y.double() - want).abs()
    assert bool((err <= bound + 2.0 ** -126).all()), float((err / (bound + 1e-300)).max())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,V", [
    (1, 64, 128), (1, 16, 1), (1, 256, 32), (16, 256, 128), (3, 100, 33), (5, 1000, 160), (17, 4096, 1000), (33, 520, 300),
    (64, 640, 8000), (65, 640, 257), (100, 72, 20000), (128, 1024, 2000), (129, 300, 515), (256, 512, 777), (257, 256, 4000),
    (300, 1111, 515), (1000, 520, 1111), (2000, 768, 5000), (513, 4096, 40)])
def test_product(fmt, dtype, N, D, V):
    h, w = _pair(N, D, V, fmt, N + D + V)
    y = flce.linear_fp4(h, w, dtype=TYPES[dtype])
    assert y.shape == (N, V) and y.dtype == TYPES[dtype]
    _check(y, h, w)
    assert torch.equal(flce.linear_fp4(h, w, dtype=TYPES[dtype]), y)
    # into a view among others, rows any distance apart, at any element
    flat = torch.full((N * (V + 3) + 9,), 5.0, dtype=TYPES[dtype], device=DEV)
    out = flat[1:1 + N * (V + 3)].view(N, V + 3)[:, :V]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert flce.linear_fp4(h, w, out=out, status=status) is out
    assert torch.equal(out, y) and flce.check_status(status) == flce.FLCE_OK
    out.fill_(5.0)
    assert bool((flat == 5.0).all())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_one_row_at_a_time(fmt):
    """Every code, sign and scale in every place of a step: a row of the product for one value of H."""
    D, V = 512, 384
    w = torch.randn(V, D, device=DEV) * torch.exp2(torch.randint(-6, 6, (V, D // 16), device=DEV).float()).repeat_interleave(16, 1)
    W = flce.quantize_fp4(w, format=fmt)
    H = flce.quantize_fp4(torch.eye(D, device=DEV) * -3.0, format=fmt)
    assert torch.equal(flce.dequantize_fp4(H), torch.eye(D, device=DEV) * -3.0)
    want = flce.dequantize_fp4(W).T * -3.0
    for rows in (1, 16, 30, 64, 128, 200, 512):
        for first in (0, 17, D - rows):
            if first + rows > D:
                continue
            h = flce.quantize_fp4(torch.eye(D, device=DEV)[first:first + rows] * -3.0, format=fmt)
            assert torch.equal(flce.linear_fp4(h, W, dtype=torch.float32), want[first:first + rows])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_tokens_do_not_depend_on_one_another(fmt):
    h, w = _pair(600, 1000, 900, fmt, 3)
    x = flce.dequantize_fp4(h)
    y = flce.linear_fp4(h, w, dtype=torch.float32)
    for a, b in ((0, 1), (5, 20), (7, 39), (100, 164), (200, 328), (300, 556), (3, 600)):
        part = flce.quantize_fp4(x[a:b].contiguous(), format=fmt)
        if torch.equal(flce.dequantize_fp4(part), x[a:b]):   # values in the format stay (nvfp4: where scales do)
            assert torch.equal(flce.linear_fp4(part, w, dtype=torch.float32), y[a:b])
        elif fmt == "mxfp4":
            raise AssertionError("values in the format did not stay")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_non_finite_blocks_are_nan_in_their_rows_alone(fmt):
    x = torch.randn(40, 520, device=DEV)
    w = torch.randn(300, 520, device=DEV)
    x[3, 100] = float("inf")
    w[129, 519] = float("nan")
    h, m = flce.quantize_fp4(x, format=fmt), flce.quantize_fp4(w, format=fmt)
    y = flce.linear_fp4(h, m, dtype=torch.float32)
    bad = torch.zeros(40, 300, dtype=torch.bool, device=DEV)
    bad[3] = True
    bad[:, 129] = True
    assert torch.equal(y.isnan(), bad)
    x[3, 100] = 0
    w[129, 519] = 0
    keep = flce.linear_fp4(flce.quantize_fp4(x, format=fmt), flce.quantize_fp4(w, format=fmt), dtype=torch.float32)
    assert torch.equal(y[~bad], keep[~bad])


def test_other_streams_and_graphs():
    x = torch.randn(70, 640, device=DEV).bfloat16()
    w = flce.quantize_fp4(torch.randn(3000, 640, device=DEV))
    want = flce.linear_fp4(flce.quantize_fp4(x), w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = flce.linear_fp4(flce.quantize_fp4(x, stream=side), w, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    buf = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = flce.linear_fp4(flce.quantize_fp4(buf), w)
        z = flce.token_logprobs(y, None, top_k=3)
    for k in range(3):
        buf.copy_(x.roll(k, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want.roll(k, 0))
        assert torch.equal(z.top_id, flce.token_logprobs(y, None, top_k=3).top_id)


@pytest.mark.parametrize("N", [3, 300])
def test_a_wait_that_runs_out(N):
    h, w = _pair(N, 8192, 4000, "nvfp4", 1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = flce.linear_fp4(h, w, dtype=torch.float32, status=status, timeout_ns=1)
    assert flce.check_status(status) == flce.FLCE_ERR_TIMEOUT
    good = flce.linear_fp4(h, w, dtype=torch.float32)
    late = y.isnan()
    assert bool(late.any()) and torch.equal(y[~late], good[~late])


def test_refusals():
    x = torch.zeros(3, 64, device=DEV)
    h, w = flce.quantize_fp4(x), flce.quantize_fp4(torch.zeros(5, 64, device=DEV))
    m = flce.quantize_fp4(x, format="mxfp4")
    cut = flce.Fp4Matrix(h.codes, h.scales[:-16], h.row_scales, h.shape, h.format)
    for call, error in (
            (lambda: flce.quantize_fp4(x, format="fp4"), ValueError), (lambda: flce.quantize_fp4(x.half()), TypeError),
            (lambda: flce.quantize_fp4(x.cpu()), ValueError), (lambda: flce.dequantize_fp4(h, dtype=torch.float16), TypeError),
            (lambda: flce.dequantize_fp4(cut), ValueError), (lambda: flce.linear_fp4(cut, w), ValueError),
            (lambda: flce.linear_fp4(h, m), ValueError), (lambda: flce.linear_fp4(h, flce.quantize_fp4(x[:, :60])), ValueError),
            (lambda: flce.linear_fp4(h, w, dtype=torch.float16), TypeError),
            (lambda: flce.linear_fp4(h, w, out=torch.zeros(3, 4, device=DEV)), ValueError),
            (lambda: flce.linear_fp4(h, w, timeout_ns=-1), flce.FLCEError),
            (lambda: flce.Fp4Matrix.from_rows(h.codes, h.block_scales()[:, :1]), ValueError),
            (lambda: flce.Fp4Matrix.from_rows(m.codes, m.block_scales(), torch.ones(3, device=DEV), format="mxfp4"), ValueError)):
        with pytest.raises(error):
            call()
