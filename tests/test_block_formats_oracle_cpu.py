"""The block-scaled formats' oracle, pinned by what the formats fix."""
import math

import numpy as np
import pytest

from oracle import block_formats as bf


def test_grids():
    assert bf.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert bf.E4M3[-1] == 448 and bf.E4M3[1] == 2.0 ** -9 and bf.E4M3[8] == 2.0 ** -6 and bf.E4M3[0x38] == 1.0
    assert (np.diff(bf.E4M3) > 0).all() and len(bf.E4M3) == 127


def test_ties_go_to_even_codes():
    assert bf.nearest_code([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, 7.0], bf.E2M1).tolist() == [
        0, 2, 2, 4, 4, 6, 6, 6, 7]
    x = np.random.default_rng(0).standard_normal(2000) * 3
    q = bf.E2M1[bf.nearest_code(x, bf.E2M1)]
    assert np.array_equal(np.abs(q - np.abs(x)), np.abs(bf.E2M1[None] - np.abs(x)[:, None]).min(axis=1))


@pytest.mark.parametrize("most", [448.0, 6.0, 2688.0])
def test_scales_are_the_smallest_powers(most):
    for amax in [1e-45, 2.0 ** -126, 1e-30, 0.1, 1.0, most, np.nextafter(most, 1e9), most * 4, 448, 6, 1e38, 3.4e38]:
        e = bf.power_of_two(amax, most)
        assert amax <= most * math.ldexp(1.0, e) and (e == -127 or amax > most * math.ldexp(1.0, e - 1))
    assert bf.power_of_two(0.0, most) == -127


@pytest.mark.parametrize("fmt", ["e4m3", "mxfp4", "nvfp4"])
def test_values_are_near_and_repeat(fmt):
    g = np.random.default_rng(1)
    x = (g.standard_normal((7, 77)) * np.exp(g.standard_normal((7, 1)) * 3)).astype(np.float32)
    x[2] = 0
    call = bf.pack_e4m3 if fmt == "e4m3" else lambda v: bf.quantize_fp4(v, fmt)
    v = call(x)[-1]
    size = 16 if fmt == "nvfp4" else 32
    for i in range(0, 77, size):
        amax = np.abs(x[:, i:i + size]).max(axis=1, keepdims=True)
        # half the largest step: 2^-4 of a value (E4M3), or a sixth of the largest (E2M1: from 4 to 6);
        # nvfp4's scale is rounded too, by 2^-4, which may cut the largest by as much
        bound = 2.0 ** -4 * np.abs(x[:, i:i + size]) + 2.0 ** -17 * amax if fmt == "e4m3" else amax * (1 / 6 + 2.0 ** -4)
        if fmt == "mxfp4":
            bound = amax / 3
        assert (np.abs(v[:, i:i + size] - x[:, i:i + size]) <= bound).all()
    if fmt != "nvfp4":   # what is in the format stays as it is
        assert np.array_equal(call(v)[-1], v)


def test_blocks_with_infinities_are_nan():
    x = np.ones((2, 70))
    x[0, 33] = np.inf
    x[1, 69] = np.nan
    for v in (bf.pack_e4m3(x)[2], bf.quantize_fp4(x, "mxfp4")[3]):
        assert np.isnan(v[0, 32:64]).all() and np.isfinite(v[0, :32]).all() and np.isfinite(v[0, 64:]).all()
        assert np.isnan(v[1, 64:]).all() and np.isfinite(v[1, :64]).all()
    v = bf.quantize_fp4(x, "nvfp4")[3]
    assert np.isnan(v[0, 32:48]).all() and np.isnan(v).sum() == 16 + 6
