"""Attention with a sliding window whose first tokens stay visible, against the formula in 64 bits.

Tolerances as in test_gpu_decode: a score is dim products summed in 32 bits; a weight has its score's
error, the exponential's and its rounding before the product with the values (22 bits); sums over the
positions add a unit each; the output adds half a unit of its type.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests import decode_ref as ref  # noqa: E402
from tests.test_gpu_decode import Batch, gen, i32  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


def plain(bt, q, scale, window, sinks):
    """out, lse, and for each output sum p |v| and the largest sum |q||k| of its scores."""
    T, hq, dim = q.shape
    g = hq // bt.hkv
    kc, vc, ks, vs = ref.code_values(bt.k), ref.code_values(bt.v), ref.f64(bt.ks), ref.f64(bt.vs)
    out, lse, mag, sc = np.zeros((T, hq, dim)), np.full((T, hq), -np.inf), np.zeros((T, hq, dim)), np.zeros((T, hq))
    for b, c in enumerate(bt.ctx):
        n = bt.cu_np[b + 1] - bt.cu_np[b]
        for i in range(n):
            p, t = c - n + i, bt.cu_np[b] + i
            pos = np.array([j for j in range(p + 1) if (window == 0 or j > p - window or j < sinks)
                            and j // bt.page < bt.table_np.shape[1] and 0 <= bt.table_np[b][j // bt.page] < bt.pages], np.int64)
            if not len(pos):
                continue
            ids, rows = bt.table_np[b][pos // bt.page], pos % bt.page
            for h in range(hq):
                kk, vv = kc[ids, h // g, rows] * ks[ids, h // g][:, None], vc[ids, h // g, rows] * vs[ids, h // g][:, None]
                s = scale * (kk @ q[t, h])
                e = np.exp(s - s.max())
                w = e / e.sum()
                out[t, h], lse[t, h] = w @ vv, s.max() + np.log(e.sum())
                mag[t, h], sc[t, h] = w @ np.abs(vv), scale * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, lse, mag, sc


def attend_and_check(bt, hq, x, window, sinks, seed=0, workspace=True, q=None):
    bt.device()
    T, most = int(bt.cu_np[-1]), max(max(bt.new), 1)
    if q is None:
        q = (1.5 * torch.randn(T, hq, bt.dim, generator=gen(seed), device="cuda")).to(ref.TORCH[x])
    lse = torch.full((T, hq), -5.0, device="cuda")
    ws = om.new_kv_workspace(bt.cache, hq, most) if workspace else None
    out = om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, most, window=window, sinks=sinks, lse=lse, workspace=ws)
    want, wl, mag, big = plain(bt, ref.f64(q), bt.dim ** -0.5, window, sinks)
    ds = (bt.dim + 16) * 2.0 ** -22 * big
    es = min(max(max(bt.ctx), 1), window + sinks + most) * 2.0 ** -23
    tol = (2 * ds + 2.0 ** -19 + es)[..., None] * mag + 1.01 * ref.UNIT[x] * np.abs(want) + ref.TINY[x] + 1e-30
    off = np.abs(ref.f64(out) - want)
    assert (off <= tol).all(), f"outputs {float((off / tol).max())} of the tolerance"
    got = lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(wl)
    assert (np.isneginf(got) == empty).all() and (ref.f64(out)[empty] == 0).all()
    tl = ds + es + 2.0 ** -20 + 2.0 ** -22 * np.abs(wl[~empty]).max(initial=0)
    assert (np.abs(got - np.where(empty, 0, wl))[~empty] <= tl[~empty]).all(), "lse"
    return out, lse, q, ws


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 32), (256, 128), (128, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (30, 4), (64, 64), (100, 65), (17, 130), (200, 1)])
def test_windows_and_first_tokens(window, sinks, dim, page, x, kind):
    """Sequences that end before, at and long after the first position that is left out."""
    ctx = [1, 4, 34, 35, 129, 265, 700]
    attend_and_check(Batch(ctx, [1, 1, 3, 1, 2, 1, 5], 2, dim, page, kind, dim + window), 6, x, window, sinks)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("workspace", [True, False])
def test_long_sequences_split(x, workspace):
    attend_and_check(Batch([9001, 3, 6000, 64], [1, 1, 4, 2], 1, 128, 64, "int8", 3), 4, x, 2100, 5, workspace=workspace)
    attend_and_check(Batch([9001, 3, 6000], [2, 1, 1], 1, 64, 16, "e4m3", 3), 8, x, 40, 1500, workspace=workspace)


def test_many_queries_of_one_sequence():
    """Row blocks whose windows begin at different places; the gap is the first query's."""
    attend_and_check(Batch([400, 90], [170, 90], 2, 128, 32, "int8", 4), 4, "bf16", 50, 3)
    attend_and_check(Batch([350, 90], [70, 31], 1, 256, 16, "e4m3", 4), 3, "f32", 40, 20)


def test_more_queries_than_tokens_and_empty_sequences():
    attend_and_check(Batch([0, 2, 0, 240], [1, 4, 3, 1], 1, 64, 16, "int8", 2), 2, "f32", 20, 3)
    attend_and_check(Batch([50, 220, 30], [0, 2, 0], 2, 64, 16, "e4m3", 2), 4, "f16", 20, 3)


def test_tables_shorter_than_the_sequence():
    """Entries outside the cache among the first pages, in the gap and in the window; positions behind the table."""
    bt = Batch([400, 360], [1, 2], 2, 128, 16, "int8", 6, width_extra=0)
    bt.table_np[0, 0], bt.table_np[1, 1] = -1, bt.pages
    bt.table_np[0, 9], bt.table_np[0, 23] = 2 ** 31 - 1, -7
    attend_and_check(bt, 4, "f32", 60, 40)
    for width in (1, 3, 8, 21):
        bt = Batch([400, 360], [1, 2], 2, 128, 16, "int8", 6, width_extra=0)
        bt.table_np = bt.table_np[:, :width]
        attend_and_check(bt, 4, "bf16", 60, 20)


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_what_the_mask_hides_does_not_count(x):
    """NaN codes and scales between the first tokens and the window, in their own pages too, and behind the end."""
    ctx, new, window, sinks = [170, 137, 300], [1, 2, 1], 20, 5
    bt = Batch(ctx, new, 2, 128, 16, "e4m3", 21)
    for b, c in enumerate(ctx):
        pid, row = bt.table_np[b][(c - 1) // 16], (c - 1) % 16
        for t in (bt.k, bt.v):
            t.view(torch.int8)[pid, :, row + 1:] = 0x7F
            t.view(torch.int8)[bt.table_np[b][0], :, sinks:] = 0x7F
        for j in range(1, (c - new[b] - window + 1) // 16):
            bt.ks[bt.table_np[b][j]] = float("nan")
            bt.vs[bt.table_np[b][j]] = float("inf")
            bt.k.view(torch.int8)[bt.table_np[b][j]] = 0x7F
    attend_and_check(bt, 4, x, window, sinks)


def test_a_first_page_that_is_not_finite_shows():
    bt = Batch([300, 300], [1, 1], 1, 64, 16, "int8", 5).device()
    q = torch.randn(2, 2, 64, device="cuda")
    bt.vs[int(bt.table_np[0][0])] = float("nan")
    bt.ks[int(bt.table_np[1][5])] = float("nan")  # in the gap
    out = om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, 1, window=50, sinks=1)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()
    out = om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, 1, window=50)
    assert torch.isfinite(out).all()


def test_nothing_to_leave_out_is_the_plain_call():
    """No window, no first tokens, or first tokens that are all the table holds."""
    bt = Batch([700, 31], [2, 1], 2, 128, 32, "int8", 5).device()
    q = torch.randn(3, 8, 128, generator=gen(1), device="cuda").bfloat16()
    ws = om.new_kv_workspace(bt.cache, 8, 2)
    call = lambda **kw: om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, 2, workspace=ws, **kw)
    everything, windowed = call(), call(window=100)
    for kw in (dict(sinks=4), dict(window=100, sinks=10 ** 6), dict(window=100, sinks=2 ** 40), dict(window=2 ** 40, sinks=4)):
        assert torch.equal(call(**kw), everything), kw
    assert torch.equal(call(window=100, sinks=0), windowed)
    assert not torch.equal(call(window=100, sinks=4), windowed)


def test_bits_repeat_and_a_graph_follows_the_lengths():
    bt = Batch([7000, 1, 3500, 2500], [1, 1, 1, 1], 2, 128, 16, "int8", 8)
    out, lse, q, ws = attend_and_check(bt, 8, "f32", 1000, 10)
    call = lambda: om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, 1, window=1000, sinks=10, workspace=ws)
    for _ in range(4):
        assert torch.equal(call(), out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    bt.lens -= i32([3000, 0, 2600, 1])
    graph.replay()
    assert torch.equal(call(), got) and not torch.equal(got, out)


def test_binding_and_library_refuse():
    bt = Batch([70, 31], [2, 1], 2, 128, 32, "int8", 5).device()
    q = torch.randn(3, 8, 128, generator=gen(1), device="cuda").bfloat16()
    with pytest.raises(om.OmError):
        om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, 2, window=5, sinks=-1)
