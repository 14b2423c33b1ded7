"""The decoding operators' refusals at the ends of 32-bit positions, on the host: nothing is launched."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_decode_api import BIG, L, MB, append, attend, cache, read  # noqa: E402, F401


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_tables_that_reach_the_end_of_32_bits(L, page):  # noqa: F811
    width = ((1 << 31) - 1) // page
    c = cache(page=page)
    assert append(L, c, width=width, bt=1 << 40) == BIG and read(L, c, width=width, bt=1 << 40) == BIG
    assert attend(L, c, width=width, bt=1 << 40) == BIG


def test_rows_that_reach_the_end_of_32_bits(L):  # noqa: F811
    assert attend(L, cache(heads=1), tokens=((1 << 31) - 1) // 4, q_ts=0) == BIG
