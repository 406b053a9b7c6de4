"""4-bit quantisation of the largest and the smallest rows that fp32 holds: row scales from 2^-126 to
2^117, every block scale, ties between codes and between scales with the values on either side of them,
bit for bit the definition."""
import numpy as np
import pytest

from oracle import block_formats as bf
from test_fp4_gpu import _row_codes
from test_layer_norm_gpu import _put

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

CODE_TIES = (bf.E2M1[1:] + bf.E2M1[:-1]) / 2
SCALE_TIES = (bf.E4M3[1:] + bf.E4M3[:-1]) / 2


def _beside(x):
    """Each x and its two neighbours in fp32."""
    with np.errstate(over="ignore"):
        x = np.asarray(x).astype(np.float32)
    return np.concatenate([x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(np.inf))])


def _check(x, dtype, fmt):
    xt, x = _put(x, dtype)
    m = flce.quantize_fp4(xt, format=fmt)
    codes, scales, rows, values = bf.quantize_fp4(x, fmt)
    if fmt == "nvfp4":
        assert np.array_equal(m.row_scales.cpu().numpy(), rows)
    assert np.array_equal(m.block_scales().cpu().numpy(), scales)
    assert np.array_equal(_row_codes(m)[:, :x.shape[1]], codes)
    with np.errstate(over="ignore"):   # 6 s g of the largest rows may be past fp32
        assert np.array_equal(flce.dequantize_fp4(m).cpu().numpy(), values.astype(np.float32))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("exponent", [117, 116, 115, 100, 97, 96, 0, -94, -95, -96, -110, -125, -126])
def test_codes_beside_ties(fmt, dtype, exponent):
    """A row whose scale is 2^exponent, with blocks of every scale s: 6 s, and 15 values at and beside ties."""
    g = np.ldexp(1.0, exponent)
    top = 2040.0 if exponent == 117 else 2688.0   # of the row; bf16 ends at 2040 2^117
    blocks = [np.concatenate([[top * g], np.zeros(15)])]
    for s in bf.E4M3[1:]:
        if s > top / 6 * 1.05:
            continue
        ties = _beside(CODE_TIES * s * g)
        for part in (ties[:15], ties[6:21]):
            blocks.append(np.concatenate([[min(6 * s, top) * g], part]))
    x = np.concatenate(blocks)[None].astype(np.float32)
    x = np.concatenate([x, -x])
    if fmt == "nvfp4" and dtype == "f32":
        assert bf.quantize_fp4(x[:, :16], fmt)[2][0] == g
    _check(x, dtype, fmt)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("exponent", [117, 116, 96, 3, -95, -96, -126])
def test_scales_beside_ties(fmt, dtype, exponent):
    """Blocks whose largest value divided by 6 is at or beside a tie between two scales."""
    g = np.ldexp(1.0, exponent)
    top = (2040.0 if exponent == 117 else 2688.0) * g
    amax = _beside(6 * SCALE_TIES * g)
    amax = np.concatenate([[np.float32(top)], amax[amax <= top]])
    x = np.zeros((amax.size, 16), np.float32)
    x[:, 5] = amax
    x[:, 9] = -amax / 3
    _check(x.reshape(1, -1), dtype, fmt)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_subnormal_numbers(fmt, dtype):
    """Largest values k 2^-149 with k / 6 2^-23 at and beside ties between scales, and the smallest ones."""
    k = (6 * SCALE_TIES[SCALE_TIES * 6 < 1] * 2.0 ** 23)[:, None] + np.arange(-4, 5)
    k = np.concatenate([k.ravel(), np.arange(1, 40)])
    x = np.zeros((k.size, 16))
    x[:, 0] = k
    x[:, 3] = np.floor(k / 2)
    x[:, 7] = -np.floor(k / 5)
    x = np.ldexp(x, -149).reshape(1, -1)
    _check(x, dtype, fmt)
    _check(np.ldexp(np.arange(1, 49.0)[None], -149), dtype, fmt)
