"""The refusals of om_kv_append_axes that om_kv_append does not have, on the host: nothing is launched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests.test_decode_api import ALIAS, ALIGN, BIG, INV, MB, NUL, OK, cache  # noqa: E402


@pytest.fixture(scope="module")
def L():
    om.build()
    return om.lib()


def append(L, tokens=5, pos=10 * MB, axes=3, stride=5, axis=11 * MB, k=2 * MB, qo=8 * MB, rot=64):
    c = cache()
    return L.om_kv_append_axes(ctypes.addressof(c), 2, tokens, 3, 4, MB, 256, 64, k, 128, 64, 3 * MB, 128, 64, 0, 4 * MB, 100, rot, 0, 5 * MB, 4, 6 * MB,
                               7 * MB, qo, 256, 64, pos, axes, stride, axis, None)


def test_append_axes_refusals(L):
    assert append(L, axes=0) == INV and append(L, axes=-1) == INV and append(L, stride=4) == INV
    assert append(L, pos=None) == INV and append(L, pos=None, axes=0) == INV  # an axis of pairs without positions
    assert append(L, axes=65536) == BIG and append(L, stride=1 << 41) == BIG
    assert append(L, pos=10 * MB + 2) == ALIGN and append(L, axis=11 * MB + 1) == ALIGN
    assert append(L, pos=16 * MB) == ALIAS and append(L, axis=48 * MB) == ALIAS  # inside the cache
    assert append(L, pos=8 * MB + 64) == ALIAS and append(L, axis=8 * MB) == ALIAS  # inside the rotated queries
    assert append(L, tokens=0) == OK and append(L, k=None) == NUL
