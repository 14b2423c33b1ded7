"""The append with rotary positions of several axes, bit for bit against the definition in 32 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests import decode_ref as ref  # noqa: E402
from tests.test_gpu_decode import Batch, bits, gen, i32  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


def turned(x, table, positions, axis, rot, interleaved):
    """ref.rotate with the row of each pair's own axis."""
    y = x.astype(np.float32).copy()
    for t in range(x.shape[0]):
        for i in range(rot // 2):
            a = 0 if axis is None else int(axis[i])
            p = int(positions[a][t]) if 0 <= a < len(positions) else -1
            c, s = table[p][i] if 0 <= p < table.shape[0] else np.full(2, np.nan, np.float32)
            one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            u, v = x[t, :, one].astype(np.float32), x[t, :, two].astype(np.float32)
            with np.errstate(invalid="ignore", over="ignore"):
                y[t, :, one] = u * c - v * s
                y[t, :, two] = v * c + u * s
    return y


def append_and_check(bt, hq, x, rot, pairs, axes, axis, seed=0, rows=60, positions=None, behind=0):
    bt.device()
    T = int(bt.cu_np[-1]) + behind
    fused = torch.randn(T, hq + 2 * bt.hkv, bt.dim, generator=gen(seed), device="cuda").to(ref.TORCH[x])
    q, k, v = fused[:, :hq], fused[:, hq:hq + bt.hkv], fused[:, hq + bt.hkv:]
    table = om.rope_table(rows, rot, base=1000.0)
    if positions is None:
        positions = np.random.default_rng(seed).integers(0, rows, (axes, T))
    as32 = lambda t: t.float().cpu().numpy()
    tab, inter = table.cpu().numpy(), pairs == "interleaved"
    want_q = torch.from_numpy(turned(as32(q), tab, positions, axis, rot, inter)).to(q.dtype)
    want = []
    for codes, scales, new in ((bt.k, bt.ks, turned(as32(k), tab, positions, axis, rot, inter)), (bt.v, bt.vs, as32(v))):
        want.append(ref.append(codes.view(torch.int8).cpu().numpy(), scales.cpu().numpy(), new, bt.table_np, bt.ctx, bt.cu_np, bt.page, bt.kind))
    # the positions lie in a wider buffer
    wide = torch.full((axes, T + 5), -77, dtype=torch.int32, device="cuda")
    wide[:, 2:T + 2] = torch.from_numpy(np.asarray(positions, np.int32)).cuda()
    got = om.kv_append(bt.cache, q, k, v, table, bt.table, bt.lens, bt.cu, max(bt.new), pairs=pairs, positions=wide[:, 2:T + 2],
                       pair_axis=None if axis is None else i32(list(axis)))
    a, b = got.float().cpu().numpy(), want_q.float().numpy()
    nan = np.isnan(b)
    assert (np.isnan(a) == nan).all() and (bits(a)[~nan] == bits(b)[~nan]).all(), "queries"
    for name, codes, scales, (wc, ws) in (("keys", bt.k, bt.ks, want[0]), ("values", bt.v, bt.vs, want[1])):
        gs = scales.cpu().numpy()
        nan = np.isnan(ws)
        assert (np.isnan(gs) == nan).all() and (bits(gs)[~nan] == bits(ws)[~nan]).all(), f"{name}: scales"
        gc = codes.view(torch.int8).cpu().numpy()
        if bt.kind == "e4m3":  # either sign of zero
            gc, wc = np.where(gc == -128, 0, gc), np.where(wc == -128, 0, wc)
        assert (gc == wc).all(), f"{name}: {int((gc != wc).sum())} codes"


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot,page,sections,order", [(64, 64, 16, (8, 12, 12), "blocks"), (128, 128, 32, (22, 21, 21), "turns"), (128, 64, 64, (31, 1), "blocks"),
                                                         (256, 24, 16, (4, 0, 8), "turns"), (128, 128, 128, (64,), "blocks")])
def test_axes_bit_for_bit(dim, rot, page, sections, order, pairs, x, kind):
    axis = om.rope_axes(sections, order).cpu().tolist()
    append_and_check(Batch([1, 17, 16, 40, 200, 33], [1, 1, 1, 3, 70, 33], 2, dim, page, kind, dim + rot), 6, x, rot, pairs, len(sections), axis)


def test_the_axes_of_pairs():
    assert om.rope_axes((2, 1, 3), device="cpu").tolist() == [0, 0, 1, 2, 2, 2]
    assert om.rope_axes((2, 1, 3), "turns", device="cpu").tolist() == [0, 1, 2, 0, 2, 2]
    for bad in ((), (3, -1)):
        with pytest.raises(ValueError):
            om.rope_axes(bad, device="cpu")
    with pytest.raises(ValueError):
        om.rope_axes((1,), "rows", device="cpu")


def test_positions_that_are_the_places_change_nothing():
    new, ctx = [1, 30, 1], [40, 70, 1]
    got = []
    for own in (False, True):
        bt = Batch(ctx, new, 2, 128, 16, "int8", 3).device()
        x = torch.randn(32, 8, 128, generator=gen(4), device="cuda").bfloat16()
        table = om.rope_table(100, 128)
        kw = {}
        if own:
            places = np.concatenate([np.arange(c - n, c) for c, n in zip(ctx, new)])
            kw = dict(positions=i32([places.tolist()] * 3), pair_axis=om.rope_axes((16, 24, 24)))
        q = om.kv_append(bt.cache, x[:, :4], x[:, 4:6], x[:, 6:], table, bt.table, bt.lens, bt.cu, 30, **kw)
        got.append((q, bt.k, bt.v, bt.ks, bt.vs))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_axes_and_positions_that_are_not_there():
    """Axes outside the given ones, positions outside the table, one axis for all pairs, the same position twice."""
    bt = lambda: Batch([40, 12], [3, 2], 2, 64, 16, "int8", 7)
    axis = [0] * 10 + [1] * 10 + [2] * 12
    append_and_check(bt(), 2, "f32", 64, "half", 2, axis)
    append_and_check(bt(), 2, "f32", 64, "half", 2, [-1] + axis[1:20] + [0] * 11 + [2 ** 31 - 1])
    positions = np.array([[0, 1, 60, 3, 59], [-1, 5, 5, 2 ** 31 - 1, 0], [7, -2 ** 31, 9, 9, 9]])
    append_and_check(bt(), 2, "f32", 64, "interleaved", 3, axis, positions=positions)
    append_and_check(bt(), 2, "bf16", 64, "half", 1, None)


def test_tokens_behind_the_last_sequence():
    """Their queries are turned by their own positions; nothing of them is stored."""
    append_and_check(Batch([40, 12], [3, 2], 2, 64, 16, "int8", 7), 2, "f32", 64, "half", 3, [0] * 8 + [1] * 12 + [2] * 12, behind=4)


def test_captured_with_positions_that_change():
    bt = Batch([20, 31], [1, 1], 2, 64, 16, "int8", 5).device()
    x = torch.randn(2, 8, 64, generator=gen(1), device="cuda")
    table, axis, pos = om.rope_table(50, 64), om.rope_axes((8, 12, 12)), i32([[3, 4], [5, 6], [7, 8]])
    keep = [t.clone() for t in (bt.k, bt.v, bt.ks, bt.vs)]
    call = lambda: om.kv_append(bt.cache, x[:, :4], x[:, 4:6], x[:, 6:], table, bt.table, bt.lens, bt.cu, 1, positions=pos, pair_axis=axis)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = call()
    pos += 11
    for t, k in zip((bt.k, bt.v, bt.ks, bt.vs), keep):
        t.copy_(k)
    graph.replay()
    got = [t.clone() for t in (q, bt.k, bt.v, bt.ks, bt.vs)]
    for t, k in zip((bt.k, bt.v, bt.ks, bt.vs), keep):
        t.copy_(k)
    assert torch.equal(call(), got[0]) and all(torch.equal(a, b) for a, b in zip((bt.k, bt.v, bt.ks, bt.vs), got[1:]))


def test_binding_refuses():
    bt = Batch([20, 31], [1, 1], 2, 64, 16, "int8", 5).device()
    x = torch.randn(2, 8, 64, generator=gen(1), device="cuda")
    table, axis, pos = om.rope_table(50, 64), om.rope_axes((8, 12, 12)), i32([[3, 4], [5, 6], [7, 8]])
    call = lambda **kw: om.kv_append(bt.cache, x[:, :4], x[:, 4:6], x[:, 6:], table, bt.table, bt.lens, bt.cu, 1, **kw)
    for kw in (dict(pair_axis=axis), dict(positions=pos[:, :1], pair_axis=axis), dict(positions=pos, pair_axis=axis[:31]), dict(positions=pos[:0], pair_axis=axis)):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(positions=pos.long()), dict(positions=pos, pair_axis=axis.long()), dict(positions=pos.cpu(), pair_axis=axis)):
        with pytest.raises(TypeError):
            call(**kw)
