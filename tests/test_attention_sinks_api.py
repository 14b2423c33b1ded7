"""The refusals of om_kv_attention_sinks, on the host: nothing is launched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests.test_decode_api import ALIAS, INV, MB, NUL, OK, UNS, cache  # noqa: E402


@pytest.fixture(scope="module")
def L():
    om.build()
    return om.lib()


def attend(L, seqs=2, tokens=5, q=MB, window=4, sinks=2, o=8 * MB, dt=0):
    c = cache()
    return L.om_kv_attention_sinks(ctypes.addressof(c), seqs, tokens, 3, 4, q, 256, 64, dt, 5 * MB, 4, 6 * MB, 7 * MB, 0.125, window, sinks, o, 256, 64,
                                   9 * MB, 64 * MB, 64 * MB, None)


def test_attention_sinks_refusals(L):
    assert attend(L, sinks=-1) == INV and attend(L, window=-1) == INV and attend(L, window=0, sinks=-5) == INV
    assert attend(L, dt=4) == UNS and attend(L, q=None) == NUL and attend(L, o=MB + 64) == ALIAS
    assert attend(L, seqs=0) == OK and attend(L, tokens=0, q=None, o=None) == OK
