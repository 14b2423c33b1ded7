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
