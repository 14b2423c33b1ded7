"""The refusals of om_kv_shared_attention, on the host: nothing is launched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests.test_decode_api import ALIAS, ALIGN, BAD_CACHES, BIG, INV, MB, NUL, OK, UNS, cache  # noqa: E402


@pytest.fixture(scope="module")
def L():
    om.build()
    return om.lib()


def attend(L, c=None, groups=1, pt=10 * MB, pwidth=3, plen=11 * MB, at=12 * MB, seqs=2, tokens=5, max_new=3, hq=4, q=MB, q_ts=256, q_hs=64, dt=0, bt=5 * MB,
           width=4, ctx=6 * MB, cu=7 * MB, o=8 * MB, o_ts=256, o_hs=64, lse=9 * MB, ws=512 * MB, ws_bytes=512 * MB):
    c = cache() if c is None else c
    return L.om_kv_shared_attention(ctypes.addressof(c), groups, pt, pwidth, plen, at, seqs, tokens, max_new, hq, q, q_ts, q_hs, dt, bt, width, ctx, cu, 0.125,
                                    o, o_ts, o_hs, lse, ws, ws_bytes, None)


def test_shared_attention_refusals(L):
    for kw, st in BAD_CACHES:
        assert attend(L, cache(**kw)) == st, kw
    assert attend(L, groups=-1) == INV and attend(L, seqs=-1) == INV and attend(L, tokens=-1) == INV and attend(L, max_new=0) == INV
    assert attend(L, hq=3) == INV and attend(L, hq=0) == INV and attend(L, dt=4) == UNS
    assert attend(L, seqs=0) == OK and attend(L, tokens=0, q=None, o=None, ws=None) == OK
    for name in ("q", "bt", "ctx", "cu", "o", "pt", "plen", "at", "ws"):
        assert attend(L, **{name: None}) == NUL, name
    assert attend(L, width=0) == INV and attend(L, pwidth=0) == INV and attend(L, q_hs=63) == INV and attend(L, o_hs=63) == INV
    for name, at in (("q", MB), ("lse", 9 * MB), ("ws", 512 * MB), ("pt", 10 * MB), ("plen", 11 * MB), ("at", 12 * MB)):
        assert attend(L, **{name: at + 2}) == ALIGN, name
    assert attend(L, ws=512 * MB + 8) == ALIGN
    assert attend(L, ws_bytes=int(L.om_kv_shared_workspace_bytes(2, 4, 64, 3, 5)) - 1) == INV
    assert attend(L, o=MB + 64) == ALIAS and attend(L, lse=8 * MB) == ALIAS and attend(L, o=16 * MB) == ALIAS and attend(L, o=10 * MB) == ALIAS
    assert attend(L, lse=12 * MB) == ALIAS and attend(L, ws=8 * MB) == ALIAS
    assert attend(L, tokens=1 << 31) == BIG and attend(L, groups=1 << 31) == BIG and attend(L, pwidth=1 << 31) == BIG
    # tiles of the prefixes past 32 bits
    assert attend(L, groups=1 << 20, pwidth=1 << 20) == BIG


def test_workspace_bytes(L):
    f = L.om_kv_shared_workspace_bytes
    small, large = f(8, 8, 128, 1, 1), f(8, 64, 128, 5, 64)
    assert L.om_kv_workspace_bytes(8, 8, 128, 1) < small < large
    assert f(3, 4, 128, 1, 1) == 0 and f(0, 0, 128, 1, 1) == 0 and f(1, 1, 128, 0, 1) == 0 and f(1, 1, 128, 1, 0) == 0 and f(1, 64, 128, 1, 1 << 31) == 0
