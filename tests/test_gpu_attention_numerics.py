"""Attention over the 8-bit cache where its numbers are hard: roundings, not-a-numbers, scales far apart.

Tolerances. An output before its rounding to the type: a score of `dim` products is 2 (dim / 16) tensor-core sums and
four roundings off, each 2^-23 of the sum of magnitudes `big`; a weight moves by twice its score's error (its own and the
sum's), 2^-20 for the exponential and 2^-20 for what of it is kept; sums over the positions add 2^-23 each.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests import decode_ref as ref  # noqa: E402
from tests.test_gpu_decode import Batch, gen  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


def attend(bt, q, window=0, workspace=True):
    bt.device()
    T, hq = q.shape[:2]
    most = max(max(bt.new), 1)
    lse = torch.full((T, hq), -5.0, device="cuda")
    ws = om.new_kv_workspace(bt.cache, hq, most) if workspace else None
    out = om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, most, window=window, lse=lse, workspace=ws)
    return out, lse


def exact(bt, q, window=0):
    with np.errstate(invalid="ignore"):
        return ref.attention(ref.f64(q), ref.code_values(bt.k), ref.code_values(bt.v), ref.f64(bt.ks), ref.f64(bt.vs), bt.table_np, bt.ctx,
                             bt.cu_np, bt.dim ** -0.5, window, bt.page)


def half_unit(want, x):
    """Half a unit in the last place of each value's type."""
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.abs(want)))
    return np.maximum(np.where(want == 0, 0.0, np.exp2(e) * ref.UNIT[x]), ref.TINY[x])


def before_rounding(bt, big, mag):
    ds = (bt.dim // 8 + 4) * 2.0 ** -23 * big
    return (2 * ds + 2.0 ** -19 + max(bt.ctx) * 2.0 ** -23)[..., None] * mag


# ------------------------------------------------------------------ roundings
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("x", ["f16", "bf16"])
def test_16_bit_outputs_are_rounded_once(x, dim, kind):
    """Outputs of 16 bits come from sums of 32 bits: no further off than half a unit and what 32-bit outputs may be."""
    bt = Batch([2, 3, 5, 9, 17, 33], [1, 1, 1, 1, 1, 2], 4, dim, 16, kind, dim)
    q = (0.02 * torch.randn(7, 16, dim, generator=gen(3), device="cuda")).to(ref.TORCH[x])
    out, _ = attend(bt, q)
    want, _, mag, big = exact(bt, q)
    tol = before_rounding(bt, big, mag)
    off = np.abs(ref.f64(out) - want)
    assert (off <= tol + half_unit(np.abs(want) + tol, x)).all(), int((off > tol + half_unit(np.abs(want) + tol, x)).sum())


# ------------------------------------------------------------------ not a number
@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("x,kind,dim", [("f32", "int8", 128), ("bf16", "e4m3", 64), ("f16", "int8", 256)])
def test_lse_of_a_query_that_is_not_a_number(x, kind, dim, workspace):
    """Its outputs and its log-sum-exp are NaN, whatever the length and the split; the other rows' are not."""
    bt = Batch([1, 64, 300, 5000], [1, 1, 2, 1], 2, dim, 16, kind, dim)
    q = torch.randn(5, 4, dim, generator=gen(2), device="cuda").to(ref.TORCH[x])
    bad = torch.zeros(5, 4, dtype=torch.bool, device="cuda")
    for t, h in ((0, 1), (1, 3), (2, 0), (4, 2)):
        q[t, h, dim - 3] = float("nan")
        bad[t, h] = True
    out, lse = attend(bt, q, workspace=workspace)
    assert (torch.isnan(out).all(-1) == bad).all() and (torch.isnan(out).any(-1) == bad).all()
    assert (torch.isnan(lse) == bad).all() and torch.isfinite(lse[~bad]).all()


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("page,ctx,at", [(64, 50, 0), (16, 64, 2), (16, 64, 0), (64, 640, 3), (128, 9000, 40), (16, 9000, 562)])
def test_lse_of_a_key_page_that_is_not_a_number(page, ctx, at, workspace):
    """The page a warp's whole range, a part of it, or a part of one block's share."""
    bt = Batch([ctx, ctx], [1, 1], 1, 128, page, "int8", ctx + page)
    bt.ks[int(bt.table_np[0][at])] = float("nan")
    q = torch.randn(2, 4, 128, generator=gen(1), device="cuda")
    out, lse = attend(bt, q, workspace=workspace)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()


def test_lse_of_rows_that_do_not_see_the_page():
    """Three drafts around the first token of a page whose key scale is NaN: the ones behind it only."""
    bt = Batch([66, 130], [4, 3], 1, 64, 64, "e4m3", 9)
    bt.ks[int(bt.table_np[0][1])] = float("nan")
    bt.ks[int(bt.table_np[1][2])] = float("nan")
    q = torch.randn(7, 8, 64, generator=gen(1), device="cuda").bfloat16()
    out, lse = attend(bt, q)
    seen = torch.tensor([0, 0, 1, 1, 0, 1, 1], dtype=torch.bool, device="cuda")[:, None]  # positions 62 .. 65, 127 .. 129
    assert (torch.isnan(out).all(-1) == seen).all() and (torch.isnan(out).any(-1) == seen).all()
    assert (torch.isnan(lse) == seen).all() and torch.isfinite(lse[~seen[:, 0]]).all()


# ------------------------------------------------------------------ scales far apart
def two_sorts(kind, dim, x, ratio, far_score, ctx=128, new=1, seed=0):
    """Pages in turn of two sorts: even ones with a value scale `ratio` times the odd ones' and scores `far_score` lower."""
    bt = Batch([ctx, ctx - 5], [new, 1], 2, dim, 16, kind, dim + seed, width_extra=0)
    near = np.concatenate([row[1::2] for row in bt.table_np])
    far = np.concatenate([row[0::2] for row in bt.table_np])
    low = -100.0 if kind == "int8" else -112.0
    raw = torch.randint(-3, 4, bt.k.shape, generator=gen(seed + 1), device="cuda").float()
    raw[torch.from_numpy(far).cuda()] = low
    bt.k = raw.to(bt.k.dtype)
    bt.ks = torch.full_like(bt.ks, 0.02)
    bt.ks[torch.from_numpy(far).cuda()] = far_score / (0.25 * -low * dim ** 0.5)
    bt.vs[torch.from_numpy(far).cuda()] = bt.vs[torch.from_numpy(far).cuda()] * ratio
    q = torch.full((new + 1, 6, dim), 0.25, device="cuda").to(ref.TORCH[x])
    return bt, q, near, far


def check_two_sorts(bt, q, x, big, what, window=0):
    out, lse = attend(bt, q, window=window)
    want, wl, mag, _ = exact(bt, q, window)
    tol = before_rounding(bt, np.full(mag.shape[:2], big), mag)
    off = np.abs(ref.f64(out) - want)
    limit = tol + half_unit(np.abs(want) + tol, x)
    assert (off <= limit).all(), f"{what}: {float((off / limit).max())} of the tolerance"
    assert (np.abs(ref.f64(lse) - wl) <= 2e-5 + 2.0 ** -20 * np.abs(wl)).all()


@pytest.mark.parametrize("x,kind,dim", [("f32", "int8", 128), ("f32", "e4m3", 64), ("f32", "int8", 256), ("bf16", "int8", 128), ("f16", "e4m3", 128)])
@pytest.mark.parametrize("ratio", [1e3, 1e5, 1e7, 1e10, 1e20, 1e-10])
def test_pages_that_do_not_count_take_no_bits(ratio, x, kind, dim):
    """All attention is on pages whose value scale is far from the others'."""
    bt, q, _, _ = two_sorts(kind, dim, x, ratio, 150.0)
    check_two_sorts(bt, q, x, 0.3, f"ratio {ratio}")  # big: 0.25 . 3 . 0.02 . dim^0.5 of the attended ones


@pytest.mark.parametrize("kind,dim", [("int8", 128), ("e4m3", 64), ("int8", 256)])
@pytest.mark.parametrize("ratio", [1e3, 1e6, 1e10, 1e16])
def test_pages_that_count_alike(ratio, kind, dim):
    """Weights smaller by as much as the value scales are larger: both sorts are half of the output."""
    bt, q, _, _ = two_sorts(kind, dim, "f32", ratio, float(np.log(ratio)))
    check_two_sorts(bt, q, "f32", float(np.log(ratio)) + 0.3, f"ratio {ratio}")


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_pages_that_another_row_sees_take_no_bits(x):
    """Four drafts and a window that ends inside the huge page for the first of them: the others do not see it."""
    bt, q, _, _ = two_sorts("int8", 128, x, 1.0, 0.5, ctx=260, new=4)
    huge = int(bt.table_np[0][2])  # positions 32 .. 47
    bt.vs[huge] = bt.vs[huge] * 1e9
    window = 257 - 48 + 1  # of the queries at 256 .. 259: the first sees 47 and on, the others 48 and on
    check_two_sorts(bt, q, x, 0.8, "window", window=window)


def test_values_of_which_the_heaviest_is_zero():
    """The first token takes nearly all of the weight and its value is 0: what is left is the sum of the small weights."""
    bt, q, _, _ = two_sorts("int8", 128, "f32", 1.0, 0.1, ctx=512)
    for b in range(2):
        first = int(bt.table_np[b][0])
        bt.v[first, :, 0] = 0
        bt.k[first, :, 0] = 100
        bt.k[first, :, 1:] = 0
        bt.ks[first] = 12.0 / (0.25 * 100 * 128 ** 0.5)  # 12 above the others
    check_two_sorts(bt, q, "f32", 12.3, "a heavy token of value 0")


# ------------------------------------------------------------------ masked codes that are not numbers
def check_with_nan(bt, q, x, window):
    out, lse = attend(bt, q, window=window)
    want, wl, mag, big = exact(bt, q, window)
    got = ref.f64(out)
    assert (np.isnan(got) == np.isnan(want)).all(), f"{int((np.isnan(got) != np.isnan(want)).sum())} outputs"
    ok = ~np.isnan(want)
    tol = before_rounding(bt, big, np.where(ok, mag, 0.0))
    assert (np.abs(got - want)[ok] <= (tol + half_unit(np.abs(want) + tol, x))[ok]).all()
    assert (np.abs(ref.f64(lse) - wl) <= 1e-4).all()
    return np.isnan(want)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hkv,hq", [(2, 2), (1, 6)])
def test_value_codes_before_the_window_in_its_first_tile(hkv, hq, dim, x):
    bt = Batch([70, 91], [1, 1], hkv, dim, 32, "e4m3", dim)
    for b, c in enumerate(bt.ctx):
        lo = c - 20
        for t in range(lo // 16 * 16, lo):
            bt.v.view(torch.int8)[int(bt.table_np[b][t // 32]), :, t % 32] = 0x7F
    q = torch.randn(2, hq, dim, generator=gen(1), device="cuda").to(ref.TORCH[x])
    assert not check_with_nan(bt, q, x, 20).any()


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hkv,hq", [(2, 2), (1, 6)])
@pytest.mark.parametrize("window", [0, 20])
def test_value_codes_that_some_rows_see(window, hkv, hq, dim, x):
    """Drafts of which the later ones see the code, and a window that has left it behind for them: the rows that see it
    are NaN in its dimension, and nothing else is."""
    bt = Batch([45, 300], [3, 5], hkv, dim, 32, "e4m3", dim)
    raw = bt.v.view(torch.int8)
    at = lambda b, t: (int(bt.table_np[b][t // 32]), slice(None), t % 32)
    for t, d, code in ((44, 3, 0x7F), (44, dim - 1, -1), (24, 17, 0x7F)):  # 24: in the window of the first two queries
        raw[at(0, t)][..., d] = code
    for t, d, code in ((297, 0, -1), (299, 33, 0x7F), (277, 8, 0x7F), (290, 5, 0x7F)):  # 290: every row's
        raw[at(1, t)][..., d] = code
    q = torch.randn(8, hq, dim, generator=gen(1), device="cuda").to(ref.TORCH[x])
    nan = check_with_nan(bt, q, x, window)
    assert nan[2, :, 3].all() and not nan[:2, :, 3].any() and nan[3:, :, 5].all()


# ------------------------------------------------------------------ scores and scales at once
def spread(pages, hkv, lo, hi, seed):
    return 10.0 ** (lo + (hi - lo) * torch.rand(pages, hkv, generator=gen(seed), device="cuda"))


def beside_heavier(bt, q, window):
    """Sum over the positions of |value| by the largest weight among the 16 neighbours: of which a weight is 2^-24 off at most."""
    qq, out = ref.f64(q), np.zeros((*q.shape[:2], bt.dim))
    k = ref.code_values(bt.k) * ref.f64(bt.ks)[:, :, None, None]
    v = np.abs(ref.code_values(bt.v) * ref.f64(bt.vs)[:, :, None, None])
    group = q.shape[1] // bt.hkv
    for b, (c, n) in enumerate(zip(bt.ctx, bt.new)):
        for i in range(n):
            t, p = int(bt.cu_np[b]) + i, c - n + i
            pos = np.arange(max(0, p - window + 1) if window else 0, p + 1)
            ids, rows = bt.table_np[b][pos // bt.page], pos % bt.page
            for h in range(q.shape[1]):
                s = k[ids, h // group, rows] @ qq[t, h] * bt.dim ** -0.5
                w = np.exp(s - s.max())
                top = np.zeros(p // 16 + 1)
                np.maximum.at(top, pos // 16, w / w.sum())
                out[t, h] = top[pos // 16] @ v[ids, h // group, rows]
    return out


def check_spread(bt, hq, x, window=0, q_size=1.5, workspace=True, heavier=False):
    q = (q_size * torch.randn(int(bt.cu_np[-1]), hq, bt.dim, generator=gen(7), device="cuda")).to(ref.TORCH[x])
    out, lse = attend(bt, q, window=window, workspace=workspace)
    want, wl, mag, big = exact(bt, q, window)
    tol = before_rounding(bt, big, mag) + (2.0 ** -24 * beside_heavier(bt, q, window) if heavier else 0.0)
    got = ref.f64(out)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol + 2 * half_unit(np.abs(want) + tol, x)).all()
    assert np.isfinite(ref.f64(lse)).all()


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("x,kind,dim,page", [("f32", "int8", 64, 16), ("f32", "e4m3", 64, 32), ("bf16", "e4m3", 256, 16), ("bf16", "int8", 128, 64)])
def test_key_and_value_scales_far_apart(x, kind, dim, page, workspace):
    """Scores that leave most weights below 2^-126, on pages whose value scales range over 10^24: a weight of 0 stays 0."""
    bt = Batch([1785, 1039, 300], [1, 3, 2], 2, dim, page, kind, dim + page)
    bt.ks = bt.ks * spread(bt.pages, 2, -4.0, 1.3, 1)
    bt.vs = bt.vs * spread(bt.pages, 2, -12.0, 12.0, 2)
    check_spread(bt, 4, x, workspace=workspace, heavier=True)
    check_spread(bt, 4, x, window=700, workspace=workspace, q_size=15.0, heavier=True)


@pytest.mark.parametrize("lo,hi", [(-37.0, -37.0), (-36.0, -30.0), (-36.0, 0.0), (-36.0, 33.0)])
@pytest.mark.parametrize("x,kind,dim", [("f32", "int8", 64), ("f32", "e4m3", 128), ("bf16", "int8", 256)])
def test_value_scales_at_the_ends_of_the_range(x, kind, dim, lo, hi):
    bt = Batch([700, 40, 5], [2, 1, 5], 1, dim, 16, kind, dim)
    bt.vs = bt.vs * spread(bt.pages, 1, lo, hi, 3)
    check_spread(bt, 3, x)
    check_spread(bt, 3, x, window=50, q_size=0.1)


def test_value_scales_that_step_through_the_range():
    """Each page's value scale 10^36 above or below the page before, and scores that make up for it."""
    bt = Batch([128, 128], [1, 1], 1, 128, 16, "int8", 3, width_extra=0)
    bt.k = torch.full_like(bt.k, 1)
    for b in range(2):
        for j, p in enumerate(bt.table_np[b]):
            high = (j + b) % 2 == 0
            bt.vs[int(p)] = 1e-36 if high else 1.0
            bt.ks[int(p)] = 80.0 / 128 ** 0.5 if high else 0.0  # 80 above, of 83 that make up for 1e36
    q = torch.ones(2, 1, 128, device="cuda")
    out, lse = attend(bt, q)
    want, wl, mag, _ = exact(bt, q)
    tol = before_rounding(bt, np.full(mag.shape[:2], 80.0), mag)
    assert (np.abs(ref.f64(out) - want) <= tol + half_unit(np.abs(want) + tol, "f32")).all()
