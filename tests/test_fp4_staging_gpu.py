"""bf16 outputs of 4-bit products leave through two places in shared memory a warp. Where a warp's share of
a tile is an odd number of boxes, one tile ends and the next begins at different places; every box has to be
what was put there."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce
    from test_fp4_gpu import _pair

DEV = "cuda:0"


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("D", [64, 256, 520])
@pytest.mark.parametrize("N", [33, 40, 48, 72, 100, 112, 200, 300, 520, 1000])
def test_boxes_of_tile_after_tile(fmt, D, N):
    """Rows of whole 16 bytes, several tiles a CTA: the fp32 outputs, which take another way out, rounded once."""
    V = 76 * 256 * (4 if N <= 300 else 2) + 8
    h, w = _pair(N, D, V, fmt, N + D)
    want = flce.linear_fp4(h, w, dtype=torch.float32).bfloat16()
    out = torch.empty(N, V, dtype=torch.bfloat16, device=DEV)
    for _ in range(4):
        out.fill_(5.0)
        assert flce.linear_fp4(h, w, out=out) is out
        assert torch.equal(out, want)
