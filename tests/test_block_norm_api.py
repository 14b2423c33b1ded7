"""The refusals of om_block_norm, on the host: nothing is launched."""
import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402

OK, INV, NUL, ALIAS, UNS, ALIGN, BIG = 0, 1, 2, 3, 4, 7, 8
MB = 1 << 20  # stand-in device addresses: validation fails before any use


@pytest.fixture(scope="module")
def L():
    om.build()
    return om.lib()


def norm(L, tokens=4, width=64, y=MB, ldy=64, dt=0, r=2 * MB, ldr=64, rt=0, g=3 * MB, ldg=64, act=0, scale=1.0, kind=0, post=1, eps=1e-6, pw=4 * MB,
         pb=5 * MB, w=6 * MB, b=7 * MB, wt=0, s=8 * MB, lds=64, o=9 * MB, ldo=64):
    return L.om_block_norm(tokens, width, y, ldy, dt, r, ldr, rt, g, ldg, act, scale, kind, post, eps, pw, pb, w, b, wt, s, lds, o, ldo, None)


def test_block_norm_refusals(L):
    assert norm(L, tokens=-1) == INV and norm(L, width=-1) == INV
    assert norm(L, dt=3) == UNS and norm(L, rt=4) == UNS and norm(L, wt=9) == UNS and norm(L, kind=2) == UNS and norm(L, act=3) == UNS
    assert norm(L, dt=1, rt=2, wt=1) == UNS and norm(L, dt=1, rt=1, wt=2) == UNS and norm(L, dt=0, rt=1) == UNS
    for bad in (float("nan"), float("inf")):
        assert norm(L, scale=bad) == INV and norm(L, eps=bad) == INV
    assert norm(L, eps=-1e-9) == INV
    assert norm(L, post=0) == INV and norm(L, s=None, o=None) == INV
    assert norm(L, tokens=0, y=None) == OK and norm(L, width=0, y=None) == OK
    assert norm(L, y=None) == NUL
    assert norm(L, width=32769, ldy=40000, lds=40000, ldo=40000, tokens=1) == BIG and norm(L, tokens=1 << 31) == BIG and norm(L, ldy=1 << 41) == BIG
    assert norm(L, lds=63) == INV and norm(L, ldo=63) == INV and norm(L, ldy=-1) == INV and norm(L, ldr=-64) == INV and norm(L, ldg=-1) == INV
    for name in ("y", "r", "g", "pw", "pb", "w", "b", "s", "o"):
        assert norm(L, **{name: 20 * MB + 2}) == ALIGN, name
    for at in (MB, 2 * MB, 3 * MB, 4 * MB, 5 * MB, 6 * MB, 7 * MB, 9 * MB):
        assert norm(L, s=at + 16) == ALIAS, at
    for at in (MB, 2 * MB, 3 * MB, 4 * MB, 5 * MB, 6 * MB, 7 * MB, 8 * MB):
        assert norm(L, o=at + 16) == ALIAS, at
    # the place of y or of the residual, but with another stride or type
    assert norm(L, s=2 * MB, lds=65) == ALIAS and norm(L, o=MB, ldo=72) == ALIAS
    assert norm(L, s=MB, o=MB) == ALIAS
    assert norm(L, dt=1, wt=1, rt=0, o=2 * MB) == ALIAS and norm(L, dt=1, wt=1, rt=0, s=MB) == ALIAS
    assert norm(L, s=3 * MB) == ALIAS  # a gate is not


def test_binding_refusals():
    t = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        om.block_norm(t, t)
