"""Attention of sequences that share prefixes, against the formula in 64 bits.

Tolerances: a score is dim products summed in 32 bits, queries held to 22 bits (f32) or as they are; a weight has its
score's error, the exponential's (2^-21 with its argument) and its rounding in two parts of 11 bits; the tensor
cores cut a sum off at every step of 16 positions, twice for two parts, which is at most 2^-22 of the sum of magnitudes
each; the parts' joins add a few units; the output adds half a unit of its type.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests import decode_ref as ref  # noqa: E402
from tests.test_gpu_decode import gen, i32  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


class Shared:
    """A cache with random contents, prefixes and a ragged batch behind them."""

    def __init__(self, prefixes, groups, ctx, new, hkv, dim, page, kind, seed, extra=1):
        g = gen(seed)
        self.prefixes, self.groups, self.ctx, self.new = list(prefixes), list(groups), list(ctx), list(new)
        used = [max(1, -(-max(c, 1) // page)) for c in list(ctx) + list(prefixes)]
        self.pages = sum(used) + 3
        order = torch.randperm(self.pages, generator=g, device="cuda").cpu().numpy()
        at, tables = 0, []
        for part in (used[:len(ctx)], used[len(ctx):]):
            t = np.full((len(part), max(part, default=1) + extra), order[-1], np.int64)
            for b, u in enumerate(part):
                t[b, :u] = order[at: at + u]
                at += u
            tables.append(t)
        self.table_np, self.ptable_np = tables
        top = ref.TOP[kind]
        mk = lambda: (torch.randn(self.pages, hkv, page, dim, generator=g, device="cuda") * top * 0.3).clamp(-top, top)
        if kind == "int8":
            self.k, self.v = (mk().round().to(torch.int8) for _ in range(2))
        else:
            self.k, self.v = (mk().to(torch.float8_e4m3fn) for _ in range(2))
        self.ks, self.vs = ((0.5 + torch.rand(self.pages, hkv, generator=g, device="cuda")) * 3.0 / top for _ in range(2))
        self.cu_np = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.kind, self.page, self.hkv, self.dim = kind, page, hkv, dim

    def device(self):
        self.table, self.lens, self.cu = i32(self.table_np.tolist()), i32(self.ctx), i32(self.cu_np.tolist())
        self.ptable = torch.from_numpy(self.ptable_np.astype(np.int32)).cuda()
        self.plen, self.at = i32(self.prefixes), i32(self.groups)
        self.cache = om.PagedKVCache(self.k, self.v, self.ks, self.vs)
        return self

    def attend(self, q, **kw):
        return om.kv_shared_attention(self.cache, q, self.ptable, self.plen, self.at, self.table, self.lens, self.cu, max(max(self.new), 1), **kw)

    def workspace(self, hq, tokens=None):
        return om.new_shared_workspace(self.cache, hq, max(max(self.new), 1), tokens or int(self.cu_np[-1]))

    def rows_of(self, table, n):
        """(page ids, rows) of a table's first n positions that are in the cache."""
        pos = np.array([t for t in range(n) if t // self.page < len(table) and 0 <= table[t // self.page] < self.pages], np.int64)
        return table[pos // self.page], pos % self.page


def plain(s, q, scale):
    T, hq, dim = q.shape
    g = hq // s.hkv
    kc, vc, ks, vs = ref.code_values(s.k), ref.code_values(s.v), ref.f64(s.ks), ref.f64(s.vs)
    out, lse, mag, sc = np.zeros((T, hq, dim)), np.full((T, hq), -np.inf), np.zeros((T, hq, dim)), np.zeros((T, hq))
    for b, c in enumerate(s.ctx):
        own = [j for j in range(len(s.prefixes)) if s.groups[j] <= b < s.groups[j + 1]]
        pid, prow = s.rows_of(s.ptable_np[own[0]], s.prefixes[own[0]]) if own else (np.zeros(0, np.int64),) * 2
        for i in range(s.new[b]):
            t = s.cu_np[b] + i
            oid, orow = s.rows_of(s.table_np[b], c - s.new[b] + i + 1)
            ids, rows = np.concatenate((pid, oid)), np.concatenate((prow, orow))
            if not len(ids):
                continue
            for h in range(hq):
                kk, vv = kc[ids, h // g, rows] * ks[ids, h // g][:, None], vc[ids, h // g, rows] * vs[ids, h // g][:, None]
                x = scale * (kk @ q[t, h])
                e = np.exp(x - x.max())
                w = e / e.sum()
                out[t, h], lse[t, h] = w @ vv, x.max() + np.log(e.sum())
                mag[t, h], sc[t, h] = w @ np.abs(vv), abs(scale) * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, lse, mag, sc


def check(s, q, out, lse, x, scale=None):
    scale = s.dim ** -0.5 if scale is None else scale
    want, wl, mag, big = plain(s, ref.f64(q), scale)
    steps = (max(s.prefixes, default=0) + max(s.ctx)) / 8 + 64
    ds = (s.dim + 16) * 2.0 ** -22 * big
    tol = (2 * ds + 2.0 ** -19 + steps * 2.0 ** -22)[..., None] * mag + 1.01 * ref.UNIT[x] * np.abs(want) + ref.TINY[x] + 1e-30
    off = np.abs(ref.f64(out) - want)
    assert (off <= tol).all(), f"outputs {float((off / tol).max())} of the tolerance"
    got = lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(wl)
    assert (np.isneginf(got) == empty).all() and (ref.f64(out)[empty] == 0).all()
    tl = ds + (steps + 64) * 2.0 ** -22 + 2.0 ** -20 + 2.0 ** -22 * np.abs(wl[~empty]).max(initial=0)
    assert (np.abs(got - np.where(empty, 0, wl))[~empty] <= tl[~empty]).all(), "lse"


def attend_and_check(s, hq, x, q=None, seed=0, scale=None):
    s.device()
    T = int(s.cu_np[-1])
    if q is None:
        q = (1.5 * torch.randn(T, hq, s.dim, generator=gen(seed), device="cuda")).to(ref.TORCH[x])
    lse = torch.full((T, hq), -5.0, device="cuda")
    ws = s.workspace(hq)
    out = s.attend(q, lse=lse, workspace=ws, **({} if scale is None else {"scale": scale}))
    check(s, q, out, lse, x, scale)
    assert om.workspace_status(ws) == 0
    return out, lse, q, ws


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 32), (256, 128), (128, 16)])
@pytest.mark.parametrize("hkv,group,seqs,prefix", [(1, 1, 1, 1), (2, 4, 3, 128), (1, 8, 20, 300), (3, 5, 4, 65)])
def test_one_prefix(hkv, group, seqs, prefix, dim, page, x, kind):
    ctx, new = [1 + 7 * b % 40 for b in range(seqs)], [1] * seqs
    attend_and_check(Shared([prefix], [0, seqs], ctx, new, hkv, dim, page, kind, dim + seqs), hkv * group, x)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("prefix", [15, 16, 127, 129, 1000, 5003])
def test_lengths_that_end_inside_a_tile(prefix, x, kind):
    attend_and_check(Shared([prefix], [0, 3], [5, 40, 1], [2, 1, 1], 2, 128, 16, kind, prefix), 8, x)


def test_many_rows():
    """More rows than one block's, the last block nearly empty; drafts of several tokens."""
    attend_and_check(Shared([700], [0, 13], [9 + b for b in range(13)], [1 + b % 5 for b in range(13)], 2, 128, 64, "int8", 5), 24, "bf16")
    attend_and_check(Shared([333], [0, 2], [150, 90], [129, 3], 1, 64, 16, "e4m3", 6), 2, "f32")
    attend_and_check(Shared([333], [0, 1], [150], [129], 1, 256, 32, "int8", 7), 1, "f16")


def test_several_prefixes():
    """Groups of different sizes and lengths, an empty one, a prefix of no tokens, sequences outside all groups."""
    for x, kind, dim in (("f32", "int8", 64), ("bf16", "e4m3", 128), ("f16", "int8", 256)):
        s = Shared([130, 0, 900, 17], [1, 4, 6, 6, 9], [3, 20, 1, 64, 5, 6, 33, 8, 9, 2], [1, 2, 1, 3, 1, 1, 4, 1, 1, 2], 2, dim, 16, kind, 11)
        attend_and_check(s, 6, x)
    # more groups than a warp's lanes, one sequence each
    n = 45
    attend_and_check(Shared([1 + 11 * b % 200 for b in range(n)], range(n + 1), [1 + b % 9 for b in range(n)], [1] * n, 1, 64, 16, "int8", 12), 4, "bf16")
    # sequences without new tokens, and a group of them
    attend_and_check(Shared([130, 60, 70], [0, 2, 3, 5], [3, 20, 7, 64, 5], [1, 0, 0, 0, 2], 2, 64, 16, "int8", 13), 4, "f32")


def test_no_prefix_at_all():
    s = Shared([], [0], [30, 9], [1, 2], 2, 64, 16, "int8", 3)
    attend_and_check(s, 4, "bf16")
    got, lse, q, _ = attend_and_check(Shared([50, 0], [2, 2, 2], [30, 9], [1, 2], 2, 64, 16, "int8", 3), 4, "f32")
    s = Shared([50, 0], [2, 2, 2], [30, 9], [1, 2], 2, 64, 16, "int8", 3).device()
    alone = torch.empty_like(lse)
    want = om.kv_attention(s.cache, q, s.table, s.lens, s.cu, 2, lse=alone, workspace=om.new_kv_workspace(s.cache, 4, 2))
    # a row's weighted mean times its sum and back: two roundings and a reciprocal
    assert torch.allclose(got, want, rtol=2.0 ** -21, atol=0) and torch.allclose(lse, alone, rtol=2.0 ** -22, atol=2.0 ** -22)


def test_sequences_that_have_nothing_of_their_own():
    """More queries than own tokens: some see the prefix alone, some nothing."""
    attend_and_check(Shared([40, 0], [0, 2, 4], [0, 2, 0, 40], [1, 4, 3, 1], 1, 64, 16, "int8", 2), 2, "f32")


def test_a_long_prefix_split_over_all_blocks():
    for x, kind in (("f32", "int8"), ("bf16", "e4m3")):
        attend_and_check(Shared([40003], [0, 2], [5, 300], [1, 2], 1, 128, 64, kind, 8), 4, x)


def test_table_entries_outside_the_cache():
    s = Shared([300, 90], [0, 2, 3], [40, 12, 30], [1, 2, 1], 2, 128, 16, "int8", 6, extra=0)
    s.ptable_np[0, 2], s.ptable_np[0, 18], s.ptable_np[1, 0] = -1, s.pages, 2 ** 31 - 1
    s.table_np[0, 1] = -5
    attend_and_check(s, 4, "f32")
    s = Shared([300, 90], [0, 2, 3], [40, 12, 30], [1, 2, 1], 2, 64, 16, "e4m3", 6, extra=0)
    s.ptable_np = s.ptable_np[:, :4]  # positions behind the table
    attend_and_check(s, 4, "bf16")
    s.ptable_np[:] = -1  # nothing of the prefixes is there
    attend_and_check(s, 4, "bf16")


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_what_is_not_seen_does_not_count(x):
    """NaN codes behind a prefix's end and scales of pages that are not there."""
    s = Shared([70, 37], [0, 1, 3], [20, 9, 33], [1, 1, 1], 2, 128, 16, "e4m3", 21)
    for table, lens in ((s.ptable_np, s.prefixes), (s.table_np, s.ctx)):
        for b, c in enumerate(lens):
            for t in (s.k, s.v):
                t.view(torch.int8)[table[b][(c - 1) // 16], :, (c - 1) % 16 + 1:] = 0x7F
    spare = int(s.ptable_np[0, -1])
    s.ks[spare] = float("nan")
    s.vs[spare] = float("inf")
    s.k.view(torch.int8)[spare] = 0x7F
    attend_and_check(s, 4, x)


def test_a_page_that_is_not_finite_shows():
    s = Shared([200, 200], [0, 2, 3], [20, 9, 33], [1, 1, 1], 1, 64, 16, "int8", 5).device()
    q = torch.randn(3, 2, 64, generator=gen(1), device="cuda")
    ws = s.workspace(2)
    for scales, bad in ((s.vs, float("nan")), (s.vs, float("inf")), (s.ks, float("nan"))):
        keep = scales.clone()
        scales[int(s.ptable_np[0][3])] = bad
        lse = torch.empty(3, 2, device="cuda")
        out = s.attend(q, lse=lse, workspace=ws)
        assert torch.isnan(out[:2]).all() and torch.isfinite(out[2]).all() and torch.isfinite(lse[2]).all()
        scales.copy_(keep)
    q[0, 0, 5] = float("nan")
    q[1, 1, 5] = float("inf")
    out = s.attend(q, workspace=ws)
    assert torch.isnan(out[0, 0]).all() and torch.isnan(out[1, 1]).all() and torch.isfinite(out[[0, 1, 2, 2], [1, 0, 0, 1]]).all()


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
def test_wide_ranges(x):
    """Large scores, values of very different scale by page, zero and negative scales, queries of very different size."""
    s = Shared([600], [0, 3], [40, 40, 40], [1, 1, 1], 1, 128, 16, "int8", 31)
    scales = 10.0 ** torch.linspace(-4, 2, s.pages, device="cuda")
    s.vs = scales[torch.randperm(s.pages, generator=gen(1), device="cuda")][:, None].contiguous()
    s.vs[int(s.ptable_np[0][0])] = 0.0
    s.ks[int(s.ptable_np[0][3])] = 0.0
    s.ks[int(s.ptable_np[0][7])] *= -1.0
    s.vs[int(s.ptable_np[0][9])] *= -1.0
    q = torch.randn(3, 4, 128, generator=gen(2), device="cuda")
    q[0] *= 30.0
    q[1] *= 1e-3
    q[2, 0] = 0.0
    q[2, 1] *= 1e4 if x == "f16" else 1e6
    if x != "f16":
        q[2, 2] *= 1e-30
    attend_and_check(s, 4, x, q=q.to(ref.TORCH[x]), scale=0.01)
    attend_and_check(s, 4, x, q=q.to(ref.TORCH[x]), scale=-0.01)


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_scales_far_apart_keep_their_bits(x):
    """The page that counts has a scale 2^-40 of another's, whose tokens weigh next to nothing (scores 60 below)."""
    s = Shared([160], [0, 1], [1], [1], 1, 64, 16, "int8", 3, extra=0)
    s.k[:] = 0
    s.vs[:] = 1.0
    small = int(s.ptable_np[0][6])
    s.vs[small] = 2.0 ** -40
    s.ks[:] = 1.0
    s.k[small, :, :, 0] = 100
    s.v[int(s.table_np[0][0])] = 0
    for j in range(10):
        if j != 6:
            s.v[int(s.ptable_np[0][j])] = 0 if j % 2 else s.v[int(s.ptable_np[0][j])]
    q = torch.zeros(1, 2, 64, device="cuda")
    q[0, :, 0] = 0.6
    attend_and_check(s, 2, x, q=q.to(ref.TORCH[x]), scale=1.0)


def test_strides_and_what_lies_beside():
    s = Shared([90], [0, 2], [40, 31], [2, 1], 2, 64, 32, "int8", 3).device()
    rows = torch.randn(3, 12, 64, generator=gen(4), device="cuda").bfloat16()
    q = rows[:, 2:10]
    outs = torch.full((3, 20, 64), 7.0, device="cuda").bfloat16()
    ws = s.workspace(8)
    s.attend(q, out=outs[:, 1:17:2], workspace=ws)
    want = s.attend(q.contiguous(), workspace=ws)
    assert torch.equal(outs[:, 1:17:2], want) and (outs[:, 0::2] == 7).all() and (outs[:, 17:] == 7).all()
    odd = torch.zeros(3 * 600 + 1, device="cuda").bfloat16()
    view = torch.as_strided(odd, (3, 8, 64), (600, 67, 1), 1)
    view.copy_(q)
    res = torch.as_strided(torch.zeros(3 * 700 + 3, device="cuda").bfloat16(), (3, 8, 64), (700, 65, 1), 3)
    assert torch.equal(s.attend(view, out=res, workspace=ws), want)


def test_tokens_that_no_sequence_owns_stay():
    s = Shared([90], [0, 2], [40, 31], [2, 1], 2, 64, 32, "int8", 3).device()
    q = torch.randn(6, 4, 64, generator=gen(4), device="cuda")
    out, lse = torch.full((6, 4, 64), 7.0, device="cuda"), torch.full((6, 4), 3.0, device="cuda")
    ws = s.workspace(4, 6)
    s.attend(q, out=out, lse=lse, workspace=ws)
    assert (out[3:] == 7).all() and (lse[3:] == 3).all()
    assert torch.equal(out[:3], s.attend(q[:3].contiguous(), workspace=ws))


def test_bits_repeat_in_a_workspace_of_other_calls():
    """The order of the parts does not depend on timing, and nothing is kept from a call."""
    s = Shared([9000, 350], [0, 3, 4], [70, 1, 350, 25], [1, 1, 2, 1], 2, 128, 16, "int8", 8)
    out, lse, q, ws = attend_and_check(s, 8, "f32")
    other = Shared([77], [0, 2], [5, 9], [1, 2], 2, 128, 16, "e4m3", 9).device()
    small = torch.randn(3, 8, 128, generator=gen(3), device="cuda")
    first = other.attend(small, workspace=ws)
    for _ in range(4):
        l2 = torch.empty_like(lse)
        assert torch.equal(s.attend(q, lse=l2, workspace=ws), out) and torch.equal(lse, l2)
        assert torch.equal(other.attend(small, workspace=ws), first)
    assert torch.equal(s.attend(q), out)  # a workspace of its own


def test_captured_and_on_another_stream():
    s = Shared([900], [0, 3], [70, 1, 35], [1, 1, 1], 2, 128, 16, "int8", 8)
    out, _, q, ws = attend_and_check(s, 8, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = s.attend(q, workspace=s.workspace(8), stream=side)
    side.synchronize()
    assert torch.equal(got, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.attend(q, workspace=ws)
    s.lens += 3
    s.plen -= 250
    graph.replay()
    assert torch.equal(s.attend(q, workspace=ws), got) and not torch.equal(got, out)


def test_offsets_that_decrease_stay_inside():
    """Unspecified outputs, but nothing else is touched and later calls are right."""
    s = Shared([200, 100], [0, 2, 3], [20, 9, 33], [1, 1, 1], 1, 64, 16, "int8", 5)
    out, lse, q, ws = attend_and_check(s, 2, "f32")
    for bad in ([3, 0, 2], [-5, 2, 900], [2, 1, 0], [0, 0, 2 ** 31 - 1]):
        om.kv_shared_attention(s.cache, q, s.ptable, s.plen, i32(bad), s.table, s.lens, s.cu, 1, workspace=ws)
    assert torch.equal(s.attend(q, workspace=ws), out) and om.workspace_status(ws) == 0


def test_offsets_past_32_bits():
    """A prefix at the far end of a cache of more than 2^32 bytes."""
    free, _ = torch.cuda.mem_get_info()
    if free < 30 << 30:
        pytest.skip("less than 30 GB of device memory free")
    page, hkv, dim = 128, 8, 128
    pages = (1 << 32) // (page * hkv * dim) + 40
    k, v = (torch.zeros(pages, hkv, page, dim, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pages, hkv, device="cuda") for _ in range(2))
    s = Shared([700], [0, 1], [60], [1], hkv, dim, page, "int8", 12, extra=0).device()
    n = s.pages
    k[-n:], v[-n:], ks[-n:], vs[-n:] = s.k, s.v, s.ks, s.vs
    big = om.PagedKVCache(k, v, ks, vs)
    q = torch.randn(1, 16, dim, generator=gen(1), device="cuda")
    far = lambda t: (t + (pages - n)).int()
    got = om.kv_shared_attention(big, q, far(s.ptable), s.plen, s.at, far(s.table), s.lens, s.cu, 1)
    assert torch.equal(got, s.attend(q))
    del k, v, big
    torch.cuda.empty_cache()


def test_empty_calls_and_refusals():
    s = Shared([90], [0, 2], [40, 31], [2, 1], 2, 64, 32, "int8", 3).device()
    q = torch.randn(3, 4, 64, device="cuda")
    assert s.attend(q[:0]).shape == (0, 4, 64)
    with pytest.raises(om.OmError):
        s.attend(q, workspace=torch.zeros(64, dtype=torch.int32, device="cuda"))
    for kw in (dict(groups=s.at[:1]), dict(prefix_len=s.plen[:0]), dict(prefix_table=s.ptable.repeat(2, 1)), dict(q=q[:, :, :32])):
        a = dict(q=q, prefix_table=s.ptable, prefix_len=s.plen, groups=s.at, block_table=s.table, ctx_len=s.lens, cu=s.cu, max_new=2)
        a.update(kw)
        with pytest.raises(ValueError):
            om.kv_shared_attention(s.cache, **a)
    with pytest.raises(TypeError):
        om.kv_shared_attention(s.cache, q, s.ptable, s.plen.long(), s.at, s.table, s.lens, s.cu, 2)
    with pytest.raises(ValueError):
        om.new_shared_workspace(s.cache, 3, 1, 4)


def long_parts(x, dim, tokens, hq, prefix, own, same_sign, seed, tiles=4):
    """One sequence of many new tokens behind a long prefix: blocks whose parts are longer than the tiles whose sums stay in tensor
    memory (`tiles`: 4 for 32-bit queries, for others 256, or 64 where parts may be longer). Pages' scales of keys grow with the position, so that maxima rise until the end; those of
    values go up and down over 10^4. Without a sign or scales of keys: every weight is the same, and errors of a sum add up."""
    s = Shared([prefix], [0, 1], [own], [tokens], 1, dim, 64, "int8", seed)
    g = gen(seed + 1)
    q = torch.randn(tokens, hq, dim, generator=g, device="cuda")
    pages = torch.from_numpy(s.ptable_np[0]).cuda()[: -(-prefix // 64)]
    if same_sign:
        s.v = torch.randint(1, 128, s.v.shape, generator=g, device="cuda").to(torch.int8)
        s.vs[:] = 0.013
        q.zero_()
    else:
        s.ks[pages, 0] = torch.linspace(0.002, 0.06, len(pages), device="cuda")
        s.vs[pages, 0] = 10.0 ** (2 * torch.sin(0.1 * torch.arange(len(pages), device="cuda")))
    q = q.to(ref.TORCH[x])
    s.device()
    lse = torch.empty(tokens, hq, device="cuda")
    out = s.attend(q, lse=lse, workspace=s.workspace(hq))
    # the formula in 64 bits, a thousand rows at a time
    pos = torch.arange(prefix, device="cuda")
    opos = torch.arange(own, device="cuda")
    otable = torch.from_numpy(s.table_np[0]).cuda()
    ids, rows = torch.cat((pages[pos // 64], otable[opos // 64])), torch.cat((pos, opos)) % 64
    k, v = (c[ids, 0, rows].double() * sc[ids, 0][:, None].double() for c, sc in ((s.k, s.ks), (s.v, s.vs)))
    at = torch.cat((pos - prefix, opos))
    scale, worst = dim ** -0.5, 0.0
    for t0 in range(0, tokens, max(1, 1024 // hq)):
        qq = q[t0: t0 + max(1, 1024 // hq)].double()
        n = qq.shape[0]
        y = scale * (qq.reshape(-1, dim) @ k.T)
        here = (own - tokens + torch.arange(t0, t0 + n, device="cuda")).repeat_interleave(hq)
        y.masked_fill_(at > here[:, None], float("-inf"))
        top = y.amax(1, keepdim=True)
        big = scale * (qq.abs().reshape(-1, dim) @ k.abs().T).amax(1, keepdim=True)
        e = torch.exp(y - top)
        total = e.sum(1, keepdim=True)
        want, mag = e @ v / total, e @ v.abs() / total
        ds = (dim + 16) * 2.0 ** -22 * big
        # cut sums: 8 steps a tile over the tiles that stay, then one rounding a fold and part; own tokens as in check()
        steps = 8 * tiles + prefix / 64 / tiles + (0 if x == "f32" else own / 8) + 64
        tol = (2 * ds + 2.0 ** -19 + steps * 2.0 ** -22) * mag + 1.01 * ref.UNIT[x] * want.abs() + ref.TINY[x] + 1e-30
        off = (out[t0: t0 + n].reshape(-1, dim).double() - want).abs()
        assert bool((off <= tol).all()), f"outputs {float((off / tol).max())} of the tolerance at tokens from {t0}"
        worst = max(worst, float((off / mag).max()))
        wl = (top + total.log()).reshape(n, hq)
        # a tile's weights are added up in 32 bits, then the tiles
        tl = ds.reshape(n, hq) + (prefix / 64 + own / 8 + 128) * 2.0 ** -22 + 2.0 ** -20 + 2.0 ** -22 * wl.abs()
        assert bool(((lse[t0: t0 + n].double() - wl).abs() <= tl).all()), "lse"
    return worst


@pytest.mark.parametrize("x,dim,tokens,hq,prefix,own,tiles", [
    ("f32", 64, 1000, 8, 8192, 1000, 4),     # cut items of some 26 tiles
    ("f32", 128, 500, 8, 20000, 700, 4),
    ("f32", 256, 333, 4, 20001, 333, 4),     # a last block of few rows
    ("f32", 64, 2500, 16, 1500, 2500, 4),    # whole items among them
    ("bf16", 128, 1024, 16, 17000, 1024, 256),
    ("f16", 64, 4096, 16, 4500, 4096, 256),
    ("f16", 64, 4096, 10, 17300, 4096, 64),  # whole items of 271 tiles
    ("bf16", 256, 2100, 10, 17300, 2100, 64),
])
def test_parts_longer_than_sums_stay(x, dim, tokens, hq, prefix, own, tiles):
    long_parts(x, dim, tokens, hq, prefix, own, False, 40 + dim, tiles)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_sums_of_one_sign(dim):
    """Before sums were taken out of tensor memory every few tiles, they were 2.5e-5 (heads of 256: 1e-4) off here."""
    worst = long_parts("f32", dim, 512, 8, 131072, 600, True, 50)
    # 32 cut steps and some 100 folds, no score error: queries are zero
    assert worst <= 2.0 ** -19 + (64 + 32 + 16) * 2.0 ** -23
