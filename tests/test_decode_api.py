"""The decoding operators' refusals, on the host: nothing is launched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from implicit_gemm_convolution_gb300 import decode  # noqa: E402

OK, INV, NUL, ALIAS, UNS, ALIGN, BIG = 0, 1, 2, 3, 4, 7, 8
MB = 1 << 20  # stand-in device addresses, a megabyte apart: validation fails before any use


@pytest.fixture(scope="module")
def L():
    om.build()
    return om.lib()


def w4(L, m=4, n=64, k=256, group=64, x=MB, ldx=None, xt=0, w=2 * MB, ldw=None, s=3 * MB, lds=None, st=0, z=None, ldz=None,
       y=4 * MB, ldy=None):
    g = -(-k // group) if group > 0 else 1
    d = lambda v, e: e if v is None else v
    return L.om_w4_matvec(m, n, k, group, x, d(ldx, k), xt, w, d(ldw, (k + 1) // 2), s, d(lds, g), st, z, d(ldz, g), y, d(ldy, n), None)


def test_w4_refusals(L):
    assert w4(L, m=-1) == INV and w4(L, n=-1) == INV and w4(L, k=-1) == INV and w4(L, group=0) == INV
    assert w4(L, xt=3) == UNS and w4(L, st=4) == UNS and w4(L, xt=9) == UNS
    for g in (16, 48, 96, 100, 160):
        assert w4(L, group=g) == UNS
    assert w4(L, m=0, x=None, w=None, s=None, y=None) == OK and w4(L, n=0, y=None) == OK
    assert w4(L, ldx=255) == INV and w4(L, ldw=127) == INV and w4(L, lds=3) == INV and w4(L, ldy=63) == INV
    assert w4(L, z=5 * MB, ldz=3) == INV
    assert w4(L, x=None) == NUL and w4(L, w=None) == NUL and w4(L, s=None) == NUL and w4(L, y=None) == NUL
    assert w4(L, x=MB + 2) == ALIGN and w4(L, y=4 * MB + 2) == ALIGN and w4(L, s=3 * MB + 1) == ALIGN
    assert w4(L, y=MB + 64) == ALIAS and w4(L, y=2 * MB) == ALIAS and w4(L, y=3 * MB + 4) == ALIAS and w4(L, z=4 * MB) == ALIAS
    assert w4(L, m=70000) == BIG and w4(L, k=1 << 40) == BIG and w4(L, ldx=1 << 50) == BIG


def cache(k=16 * MB, v=32 * MB, ks=48 * MB, vs=49 * MB, pages=8, heads=2, page=16, dim=64, dtype=3):
    return decode._CacheStruct(k, v, ks, vs, pages, heads, page, dim, dtype)


BAD_CACHES = [(dict(pages=-1), INV), (dict(heads=0), INV), (dict(dtype=0), UNS), (dict(page=8), UNS), (dict(page=48), UNS),
              (dict(dim=96), UNS), (dict(k=None), NUL), (dict(vs=None), NUL), (dict(k=16 * MB + 8), ALIGN),
              (dict(ks=48 * MB + 2), ALIGN), (dict(pages=1 << 40), BIG)]


def append(L, c=None, seqs=2, tokens=5, max_new=3, hq=4, q=MB, q_ts=256, q_hs=64, k=2 * MB, k_ts=128, k_hs=64, v=3 * MB, v_ts=128,
           v_hs=64, dt=0, table=4 * MB, rows=100, rot=64, pairs=0, bt=5 * MB, width=4, ctx=6 * MB, cu=7 * MB, qo=8 * MB, o_ts=256,
           o_hs=64):
    c = cache() if c is None else c
    return L.om_kv_append(ctypes.addressof(c) if c else None, seqs, tokens, max_new, hq, q, q_ts, q_hs, k, k_ts, k_hs, v, v_ts, v_hs,
                          dt, table, rows, rot, pairs, bt, width, ctx, cu, qo, o_ts, o_hs, None)


def test_append_refusals(L):
    for kw, st in BAD_CACHES:
        assert append(L, cache(**kw)) == st, kw
    assert L.om_kv_append(None, *[0] * 4, *[None, 0, 0] * 3, 0, None, 0, 0, 0, None, 0, None, None, None, 0, 0, None) == NUL
    assert append(L, seqs=-1) == INV and append(L, tokens=-1) == INV and append(L, max_new=0) == INV
    assert append(L, dt=3) == UNS and append(L, rot=65) == INV and append(L, rot=12) == UNS and append(L, rot=128) == INV
    assert append(L, pairs=2) == INV
    assert append(L, seqs=0) == OK and append(L, tokens=0, q=None, k=None) == OK
    for name in ("q", "k", "v", "table", "bt", "ctx", "cu", "qo"):
        assert append(L, **{name: None}) == NUL, name
    assert append(L, width=0) == INV and append(L, k_hs=32) == INV and append(L, q_ts=-1) == INV and append(L, o_ts=255) == INV
    assert append(L, k=2 * MB + 2) == ALIGN and append(L, table=4 * MB + 4) == ALIGN and append(L, cu=7 * MB + 2) == ALIGN
    assert append(L, cache(v=16 * MB + 64)) == ALIAS and append(L, k=16 * MB) == ALIAS and append(L, bt=48 * MB) == ALIAS
    assert append(L, qo=MB + 64) == ALIAS and append(L, qo=2 * MB) == ALIAS and append(L, qo=4 * MB) == ALIAS
    assert append(L, seqs=1 << 32) == BIG and append(L, width=1 << 31) == BIG


def attend(L, c=None, seqs=2, tokens=5, max_new=3, hq=4, q=MB, q_ts=256, q_hs=64, dt=0, bt=5 * MB, width=4, ctx=6 * MB, cu=7 * MB,
           window=0, o=8 * MB, o_ts=256, o_hs=64, lse=9 * MB, ws=64 * MB, ws_bytes=64 * MB):
    c = cache() if c is None else c
    return L.om_kv_attention(ctypes.addressof(c), seqs, tokens, max_new, hq, q, q_ts, q_hs, dt, bt, width, ctx, cu, 0.125, window, o, o_ts,
                             o_hs, lse, ws, ws_bytes, None)


def test_attention_refusals(L):
    for kw, st in BAD_CACHES:
        assert attend(L, cache(**kw)) == st, kw
    assert attend(L, seqs=-1) == INV and attend(L, tokens=-1) == INV and attend(L, max_new=0) == INV and attend(L, window=-1) == INV
    assert attend(L, hq=3) == INV and attend(L, hq=0) == INV and attend(L, dt=4) == UNS
    assert attend(L, seqs=0) == OK and attend(L, tokens=0, q=None, o=None) == OK
    for name in ("q", "bt", "ctx", "cu", "o"):
        assert attend(L, **{name: None}) == NUL, name
    assert attend(L, q_hs=63) == INV and attend(L, o_hs=63) == INV and attend(L, width=0) == INV
    assert attend(L, q=MB + 2) == ALIGN and attend(L, lse=9 * MB + 2) == ALIGN and attend(L, ws=64 * MB + 8) == ALIGN
    assert attend(L, ws_bytes=int(L.om_kv_workspace_bytes(2, 4, 64, 3)) - 1) == INV
    assert attend(L, o=MB + 64) == ALIAS and attend(L, lse=8 * MB) == ALIAS and attend(L, ws=0 * MB + 16, ws_bytes=80 * MB) == ALIAS
    assert attend(L, o=16 * MB) == ALIAS and attend(L, lse=7 * MB) == ALIAS
    assert attend(L, tokens=1 << 31) == BIG


def read(L, c=None, seqs=2, tokens=5, bt=5 * MB, width=4, start=6 * MB, cu=7 * MB, k=8 * MB, v=9 * MB, dt=0):
    c = cache() if c is None else c
    return L.om_kv_read(ctypes.addressof(c), seqs, tokens, bt, width, start, cu, k, v, dt, None)


def test_read_refusals(L):
    for kw, st in BAD_CACHES:
        assert read(L, cache(**kw)) == st, kw
    assert read(L, seqs=-1) == INV and read(L, tokens=-1) == INV and read(L, dt=3) == UNS and read(L, width=0) == INV
    assert read(L, seqs=0, k=None) == OK and read(L, tokens=0, v=None) == OK
    for name in ("bt", "start", "cu", "k", "v"):
        assert read(L, **{name: None}) == NUL, name
    assert read(L, k=8 * MB + 8) == ALIGN and read(L, v=8 * MB) == ALIAS and read(L, k=16 * MB) == ALIAS and read(L, k=5 * MB) == ALIAS


def test_rope_table_refusals(L):
    f = lambda rows=4, rot=8, base=1e4, scaling=0, factor=1.0, orig=0.0, fast=32.0, slow=1.0, t=MB: L.om_rope_table(
        rows, rot, base, scaling, factor, orig, fast, slow, t, None)
    assert f(rows=-1) == INV and f(rot=3) == INV and f(rot=0) == INV and f(base=1.0) == INV and f(factor=0.5) == INV
    assert f(base=float("nan")) == INV and f(factor=float("nan")) == INV
    assert f(scaling=4) == UNS and f(scaling=3, orig=0.0) == INV and f(scaling=3, orig=100.0, fast=1.0) == INV
    assert f(t=None) == NUL and f(t=MB + 2) == ALIGN and f(rows=0, t=None) == OK and f(rows=1 << 40) == BIG


def test_parts_of_one_buffer_that_overlap(L):
    """Rotated queries beside keys and values of the same rows (parts that do not overlap
    pass: the append in place on the GPU)."""
    ts = 8 * 64  # q, k, v rows of one buffer: 4 + 2 + 2 heads of 64
    at = lambda head: MB + 4 * 64 * head
    kw = dict(q=at(0), q_ts=ts, k=at(4), k_ts=ts, v=at(6), v_ts=ts, o_ts=ts)
    assert append(L, qo=at(1), **kw) == ALIAS
    assert append(L, qo=at(4), **kw) == ALIAS


def test_workspace_bytes(L):
    small, large = L.om_kv_workspace_bytes(8, 8, 128, 1), L.om_kv_workspace_bytes(8, 64, 128, 5)
    assert 0 < small < large
    assert L.om_kv_workspace_bytes(3, 4, 128, 1) == 0 and L.om_kv_workspace_bytes(0, 0, 128, 1) == 0
    assert L.om_kv_workspace_bytes(1, 1, 128, 1 << 40) == L.om_kv_workspace_bytes(1, 64, 128, 64)


def test_binding_refuses_what_is_not_a_cuda_tensor():
    t = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        om.w4_matvec(t, t, t)
    with pytest.raises(TypeError):
        om.PagedKVCache(*[torch.zeros(2, 2, 16, 64, dtype=torch.int8)] * 2, *[torch.zeros(2, 2)] * 2)
