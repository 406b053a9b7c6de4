"""Token ids of any integer type as int32: what int32 does not hold stays out of every range."""
import pytest

torch = pytest.importorskip("torch")

import linear_cross_entropy_flce_gb300 as flce
from linear_cross_entropy_flce_gb300._binding import int32_ids

LEAST, MOST = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("ignore", [-100, -1, 0, LEAST, MOST])
def test_ids(ignore):
    held = [0, 5, -1, -100, 2 ** 30, MOST, LEAST]
    far = [2 ** 32 + 5, 2 ** 32 + ignore, ignore - 2 ** 32, 2 ** 31, LEAST - 1, 2 ** 62, -2 ** 63]
    got = int32_ids(torch.tensor(held + far), ignore)
    assert got.dtype == torch.int32 and got[:len(held)].tolist() == held
    for v in got[len(held):].tolist():
        assert v != ignore and not 0 <= v < MOST


def test_other_types():
    t = torch.tensor([1, 2], dtype=torch.int32)
    assert int32_ids(t, -100) is t
    for dtype in (torch.uint8, torch.int8, torch.int16, torch.uint32):
        assert int32_ids(torch.tensor([1, 2], dtype=dtype), -100).tolist() == [1, 2]
    far = int32_ids(torch.tensor([2 ** 32 - 100, 2 ** 31], dtype=torch.uint32), -100)   # not -100
    assert far.tolist() == [MOST, MOST]


def test_ignore_index_past_32_bits_is_refused():
    for i in (LEAST, MOST, -100):
        assert flce.make_options(ignore_index=i).ignore_index == i
    for i in (2 ** 32 - 100, 2 ** 31, LEAST - 1):
        with pytest.raises(ValueError):
            flce.make_options(ignore_index=i)
