"""4-bit quantisation of rows too long for the registers, which are read twice, wherever they begin: the
largest value of a row among its last 256 ones counts for the row's scale and the blocks'."""
import numpy as np
import pytest

from oracle import block_formats as bf
from test_fp4_gpu import _row_codes
from test_layer_norm_gpu import _put

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,pad,shift", [
    (16385, 0, 0), (16401, 0, 0), (16416, 1, 1), (16640, 3, 0), (16641, 0, 1), (20001, 0, 0), (20001, 7, 3), (40001, 0, 0),
    (32768, 1, 0), (32769, 0, 0), (33024, 0, 0), (40000, 0, 0)])
def test_largest_among_the_last(fmt, dtype, D, pad, shift):
    N = 5
    g = np.random.Generator(np.random.Philox(np.random.SeedSequence([D, pad, shift])))
    x = g.standard_normal((N, D))
    for r, back in enumerate((1, 2, 17, 100, 256)):   # 128 times the others, so that it alone decides
        x[r, D - back] = (1 - 2 * (r % 2)) * (500.0 + r)
    xt, x = _put(x, dtype, pad, shift)
    m = flce.quantize_fp4(xt, format=fmt)
    codes, scales, rows, values = bf.quantize_fp4(x, fmt)
    if fmt == "nvfp4":
        assert np.array_equal(m.row_scales.cpu().numpy(), rows)
    assert np.array_equal(m.block_scales().cpu().numpy(), scales)
    got = _row_codes(m)
    assert np.array_equal(got[:, :D], codes) and not got[:, D:].any()
    assert np.array_equal(flce.dequantize_fp4(m).cpu().numpy(), values.astype(np.float32))
