"""4-bit matrices whose codes and scales lie row by row, as checkpoints hold them: no rows, one value, odd
widths, and what is not taken."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("N", [0, 1, 127, 128, 129])
@pytest.mark.parametrize("D", [1, 16, 40, 63, 256, 257, 1000])
def test_there_and_back(fmt, N, D):
    m = flce.quantize_fp4(torch.randn(N, D, device=DEV), format=fmt)
    blocks = -(-D // (16 if fmt == "nvfp4" else 32))
    scales = m.block_scales()
    assert scales.shape == (N, blocks) and scales.dtype == torch.uint8
    n = flce.Fp4Matrix.from_rows(m.codes[:, :(D + 1) // 2], scales, m.row_scales, width=D, format=fmt)
    assert n.shape == (N, D) and torch.equal(n.codes, m.codes) and torch.equal(n.scales, m.scales)
    assert m.row_scales is None and n.row_scales is None or torch.equal(n.row_scales, m.row_scales)
    assert torch.equal(flce.dequantize_fp4(n), flce.dequantize_fp4(m))
    w = flce.quantize_fp4(torch.randn(5, D, device=DEV), format=fmt)
    assert torch.equal(flce.linear_fp4(n, w), flce.linear_fp4(m, w))


def test_row_scales():
    m = flce.quantize_fp4(torch.randn(3, 64, device=DEV))

    def rows(scales):
        return flce.Fp4Matrix.from_rows(m.codes, m.block_scales(), scales).row_scales

    one = torch.ones(3, device=DEV)
    assert torch.equal(rows(None), one) and torch.equal(rows(0.25), one / 4) and torch.equal(rows(one[:1] * 3), one * 3)
    assert torch.equal(rows(one.sum()), one * 3) and torch.equal(rows(m.row_scales), m.row_scales)
    assert torch.equal(rows(torch.arange(3)), torch.arange(3.0, device=DEV))
    for wrong in (one[:, None], one[:2], torch.ones(4, device=DEV), one[None]):
        with pytest.raises(ValueError):
            rows(wrong)
    w = rows(one)
    w.zero_()   # its own memory
    assert bool((one == 1).all())
