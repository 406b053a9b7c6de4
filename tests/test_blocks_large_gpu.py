"""The block-scaled formats past 2^31 elements and bytes: rows far into a large matrix are what they are alone."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"
SIZES = [(140_003, 16_400), (280_003, 8_192), (280_003, 8_001)]   # 2.2e9 values and more


def _far(N, D):
    return [0, 1, N // 2, 2 ** 31 // D, 2 ** 31 // D + 1, N - 4, N - 1]


def _rows(N, D):
    x = torch.zeros(N, D, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    for r in _far(N, D):
        x[r] = torch.randn(D, generator=g, device=DEV)
    return x


@pytest.mark.parametrize("N,D", SIZES)
def test_packed_rows_and_the_norm_of_them(N, D):
    x = _rows(N, D)
    p = flce.pack_e4m3(x)
    r, q = flce.layer_norm_packed(x)
    back = flce.unpack_e4m3(p)
    for i in _far(N, D):
        one = flce.pack_e4m3(x[i:i + 1])
        assert torch.equal(p.data[i], one.data[0]) and torch.equal(q.data[i], one.data[0])
        assert torch.equal(back[i], flce.unpack_e4m3(one)[0])
    del back, p
    dx, dw, _ = flce.layer_norm_packed_backward(x, q, None, r)
    # alone and among others: other orders of the sums move an element over one rounding to bf16 at most, a step of
    # 2^-5 for |y| below 8; and dx, of x - x~ (2^-4 of x), by one of 2^-8 below 1
    for i in _far(N, D):
        few, kept = flce.layer_norm_packed(x[i:i + 1])
        want = flce.layer_norm_packed_backward(x[i:i + 1], kept, None, few)[0][0]
        assert float(few.y.float().abs().max()) < 8 and float(want.float().abs().max()) < 1
        assert float((r.y[i].float() - few.y[0].float()).abs().max()) <= 2.0 ** -5
        assert float((dx[i].float() - want.float()).abs().max()) <= 2.0 ** -8
    assert float(r.y[2].float().abs().max()) == 0 and bool(torch.isfinite(dw).all())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("N,D", SIZES)
def test_4_bit_rows(fmt, N, D):
    x, far = _rows(N, D), _far(N, D)
    m = flce.quantize_fp4(x, format=fmt)
    back = flce.dequantize_fp4(m, dtype=torch.bfloat16)
    for i in far:
        one = flce.quantize_fp4(x[i:i + 1], format=fmt)
        assert torch.equal(m.codes[i], one.codes[0])
        assert torch.equal(back[i], flce.dequantize_fp4(one, dtype=torch.bfloat16)[0])
    assert bool((back[2] == 0).all()) and bool((back[N - 2] == 0).all())
    h = flce.quantize_fp4(x[far].contiguous(), format=fmt)   # and as a weight of many rows
    y = flce.linear_fp4(h, m, dtype=torch.float32)
    w = flce.linear_fp4(h, h, dtype=torch.float32)
    assert torch.equal(y[:, far], w)
    y[:, far] = 0
    assert bool((y == 0).all())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype,V", [("bfloat16", 120_000), ("bfloat16", 120_001), ("float32", 120_000)])
def test_products(fmt, dtype, V):
    rows, d = 18_001, 64   # 2.16e9 outputs
    g = torch.Generator(device=DEV).manual_seed(V)
    h = flce.quantize_fp4(torch.randn(rows, d, generator=g, device=DEV), format=fmt)
    w = flce.quantize_fp4(torch.randn(V, d, generator=g, device=DEV), format=fmt)
    y = flce.linear_fp4(h, w, dtype=getattr(torch, dtype))
    for first in (0, 9_000, 17_880, rows - 40):   # past element 2^31 from row 17895 on
        part = flce.Fp4Matrix.from_rows(h.codes[first:first + 40], h.block_scales()[first:first + 40],
                                        None if h.row_scales is None else h.row_scales[first:first + 40], width=d, format=fmt)
        assert torch.equal(flce.linear_fp4(part, w, dtype=getattr(torch, dtype)), y[first:first + 40])
