"""The decoding operators on the GPU against plain references: the 4-bit
product, the append to the paged 8-bit cache, attention over it and its read back.

Tolerances follow from the arithmetic. Sums of n terms in 32 bits are within
n 2^-23 of the sum of magnitudes (the tensor cores' sums are not rounded to
nearest, hence twice the unit); a result rounded to its type adds half a unit.
Appended codes, scales, rotated queries and values read back have one bit pattern
and are compared bit for bit.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests import decode_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------- 4-bit product
def w4_inputs(m, n, k, group, x, zeros, seed, scale_type=None):
    g = gen(seed)
    groups = -(-k // group)
    X = torch.randn(m, k, generator=g, device="cuda").to(ref.TORCH[x])
    U = torch.randint(0, 256, (n, (k + 1) // 2), dtype=torch.uint8, generator=g, device="cuda")
    S = (0.01 + 0.02 * torch.rand(n, groups, generator=g, device="cuda")).to(ref.TORCH[scale_type or x])
    Z = torch.randint(0, 16, (n, groups), dtype=torch.uint8, generator=g, device="cuda") if zeros else None
    return X, U, S, Z


def check_w4(y, X, U, S, Z, k, group, x, what=""):
    w = ref.w4_weights(U, S, Z, k, group)
    xx = ref.f64(X)
    want, mag = xx @ w.T, np.abs(xx) @ np.abs(w).T
    # per term: the sum's rounding; the scale's product and the joining of groups and
    # splits add a few more
    tol = (k + 64) * 2.0 ** -23 * mag + 1.01 * ref.UNIT[x] * np.abs(want) + ref.TINY[x]
    off = np.abs(ref.f64(y) - want)
    assert (off <= tol).all(), f"{what}: {float((off / np.maximum(tol, 1e-300)).max())} of the tolerance"


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k,group,zeros", [
    (1, 64, 256, 128, False), (1, 1, 1, 32, False), (1, 17, 33, 32, True), (2, 100, 300, 64, True),
    (3, 16, 4096, 128, False), (5, 130, 1000, 256, True), (8, 257, 511, 32, True), (9, 48, 640, 640, False),
    (16, 96, 2047, 64, False), (17, 33, 129, 128, True), (40, 20, 96, 32, False), (1, 300, 20000, 128, True),
    (7, 31, 8192, 1024, False), (65, 70, 130, 128, True),
])
def test_w4_matches_the_formula(m, n, k, group, zeros, x):
    X, U, S, Z = w4_inputs(m, n, k, group, x, zeros, 7 * m + n + k)
    check_w4(om.w4_matvec(X, U, S, zeros=Z, group=group), X, U, S, Z, k, group, x)


@pytest.mark.parametrize("scale_type", ["f32", "f16", "bf16"])
def test_w4_scale_types_differ_from_the_activations(scale_type):
    X, U, S, Z = w4_inputs(3, 50, 500, 64, "bf16", True, 5, scale_type)
    check_w4(om.w4_matvec(X, U, S, zeros=Z, group=64), X, U, S, Z, 500, 64, "bf16")


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("shift,pad", [(0, 16), (16, 32), (4, 20), (1, 3), (3, 16), (16, 4)])
def test_w4_strides_and_alignments(x, shift, pad):
    """Rows of x, weights, scales, zeros and y inside wider buffers, at every alignment."""
    m, n, k, group = 4, 77, 384, 64
    X, U, S, Z = w4_inputs(m, n, k, group, x, True, 11)
    wide_u = torch.zeros(n * (k // 2 + pad) + shift, dtype=torch.uint8, device="cuda")
    u = torch.as_strided(wide_u, (n, k // 2), (k // 2 + pad, 1), shift)
    u.copy_(U)
    xw = torch.full((m, k + 5), float("nan"), dtype=X.dtype, device="cuda")
    xw[:, 1:k + 1] = X
    sw = torch.full((n, 9), float("nan"), dtype=S.dtype, device="cuda")
    sw[:, 2:8] = S
    zw = torch.full((n, 7), 255, dtype=torch.uint8, device="cuda")
    zw[:, 1:] = Z
    yw = torch.full((m, n + 3), -7.0, dtype=X.dtype, device="cuda")
    om.w4_matvec(xw[:, 1:k + 1], u, sw[:, 2:8], zeros=zw[:, 1:], group=group, out=yw[:, 2:n + 2])
    check_w4(yw[:, 2:n + 2], X, U, S, Z, k, group, x)
    assert (yw[:, :2] == -7).all() and (yw[:, n + 2:] == -7).all()


def test_w4_special_values():
    """Infinities and NaN reach exactly the rows of x that hold them; large and
    subnormal activations keep 32 bits; garbage behind an odd k does not count."""
    m, n, k, group = 6, 40, 257, 128
    X, U, S, Z = w4_inputs(m, n, k, group, "f32", False, 3)
    U[:, 0] = 0x1F  # codes 15 and 1: neither is the zero point
    X[1, 0] = float("inf")
    X[2, 1] = float("nan")
    X[3] *= 2.0 ** 120
    X[4] *= 2.0 ** -126
    X[5, :] = 0.0
    X[5, 0] = 3.0e38
    S = S * 0.01
    y = om.w4_matvec(X, U, S, group=group)
    assert torch.isinf(y[1]).all() and (y[1] > 0).all()
    assert torch.isnan(y[2]).all()
    rows = [0, 3, 5]
    check_w4(y[rows], X[rows], U, S, Z, k, group, "f32")
    w = ref.w4_weights(U, S, Z, k, group)
    want = ref.f64(X[4:5]) @ w.T
    # at 2^-126 each term's unit is the smallest subnormal's
    assert (np.abs(ref.f64(y[4:5]) - want) <= (k + 64) * 2.0 ** -149 + (k + 64) * 2.0 ** -23 * (np.abs(ref.f64(X[4:5])) @ np.abs(w).T)).all()


def test_w4_empty_and_zero_k():
    z = torch.empty(0, 0, device="cuda")
    X, U, S, _ = w4_inputs(2, 8, 64, 32, "f32", False, 1)
    assert om.w4_matvec(X[:0], U, S, group=32).shape == (0, 8)
    y = om.w4_matvec(torch.empty(2, 0, device="cuda"), torch.empty(8, 0, dtype=torch.uint8, device="cuda"),
                     torch.empty(8, 0, device="cuda"), group=32)
    assert (y == 0).all() and y.shape == (2, 8)
    del z


def test_w4_repeats_bit_for_bit_and_runs_on_its_stream():
    X, U, S, Z = w4_inputs(4, 3000, 4000, 64, "f32", True, 9)
    a = om.w4_matvec(X, U, S, zeros=Z, group=64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = om.w4_matvec(X, U, S, zeros=Z, group=64, stream=side)
    side.synchronize()
    assert torch.equal(a, b)
    assert om.device_status() == 0


# ------------------------------------------------------------------- cache
class Batch:
    """A cache with random contents and a ragged batch over it."""

    def __init__(self, ctx, new, hkv, dim, page, kind, seed, width_extra=1, shuffle=True):
        g = gen(seed)
        self.ctx, self.new = list(ctx), list(new)
        used = [max(1, -(-max(c, 1) // page)) for c in ctx]
        self.pages = sum(used) + 2
        order = torch.randperm(self.pages, generator=g, device="cuda").cpu().numpy() if shuffle else np.arange(self.pages)
        width = max(used) + width_extra
        self.table_np = np.zeros((len(ctx), width), np.int64)
        at = 0
        for b, u in enumerate(used):
            self.table_np[b, :u] = order[at: at + u]
            at += u
        self.spare = order[at:]
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
        self.cache = om.PagedKVCache(self.k, self.v, self.ks, self.vs)
        return self


def attend_and_check(bt, hq, x, window=0, scale=None, seed=0, workspace=True, q=None, what=""):
    bt.device()
    T = int(bt.cu_np[-1])
    most = max(max(bt.new), 1)
    if q is None:
        q = (1.5 * torch.randn(T, hq, bt.dim, generator=gen(seed), device="cuda")).to(ref.TORCH[x])
    lse = torch.full((T, hq), -5.0, device="cuda")
    ws = om.new_kv_workspace(bt.cache, hq, most) if workspace else None
    out = om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, most, scale=scale, window=window, lse=lse, workspace=ws)
    sc = bt.dim ** -0.5 if scale is None else scale
    want, wl, mag, big = ref.attention(ref.f64(q), ref.code_values(bt.k), ref.code_values(bt.v), ref.f64(bt.ks), ref.f64(bt.vs),
                                       bt.table_np, bt.ctx, bt.cu_np, sc, window, bt.page)
    # a score: dim products summed in 32 bits, q held to 22 bits, four roundings of factors
    ds = (bt.dim + 16) * 2.0 ** -22 * big
    # a weight: its score, the exponential (2^-21 with its argument), and its rounding before
    # the product with the values: 11 bits for 16-bit types, 22 for 32-bit ones
    ew = 2 * ds + 2.0 ** -20 + (2.0 ** -20 if x == "f32" else 2.0 ** -10)
    longest = max(max(bt.ctx), 1)
    es = longest * 2.0 ** -23  # sums over the positions
    tol = (ew + es)[..., None] * mag + 1.01 * ref.UNIT[x] * np.abs(want) + ref.TINY[x] + 1e-30
    off = np.abs(ref.f64(out) - want)
    assert (off <= tol).all(), f"{what}: outputs {float((off / tol).max())} of the tolerance"
    got = lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(wl)
    assert (np.isneginf(got) == empty).all(), f"{what}: empty rows"
    assert (ref.f64(out)[empty] == 0).all()
    tl = ds + es + 2.0 ** -20 + 2.0 ** -22 * np.abs(wl[~empty]).max(initial=0)
    assert (np.abs(got - np.where(empty, 0, wl))[~empty] <= tl[~empty]).all(), f"{what}: lse"
    return out, lse, q, ws


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hkv,group", [(1, 1), (2, 4), (1, 8), (1, 12), (3, 5), (1, 33)])
def test_attention_single_tokens(hkv, group, dim, x, kind):
    ctx = [1, 2, 15, 16, 17, 40, 200]
    attend_and_check(Batch(ctx, [1] * len(ctx), hkv, dim, 16, kind, dim + group), hkv * group, x)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("window", [0, 1, 7, 50, 128])
def test_attention_ragged_queries_pages_and_windows(page, window):
    ctx, new = [5, 130, 64, 33, 1, 300], [5, 3, 1, 9, 1, 2]
    for kind, x, dim in (("int8", "f32", 128), ("e4m3", "bf16", 64)):
        attend_and_check(Batch(ctx, new, 2, dim, page, kind, page + window), 6, x, window=window)


def test_attention_many_queries_of_one_sequence():
    """More query rows than a block holds at once."""
    attend_and_check(Batch([150, 90], [70, 90], 2, 128, 32, "int8", 4), 4, "bf16")
    attend_and_check(Batch([150, 90], [70, 31], 1, 256, 16, "e4m3", 4), 3, "f32", window=40)


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("seqs,ctx,x,kind", [(1, 9001, "f32", "int8"), (2, 5000, "bf16", "e4m3"), (3, 4097, "f16", "int8")])
def test_attention_split_sequences(seqs, ctx, x, kind, workspace):
    """Few long sequences among short ones: split over blocks with a workspace."""
    lens = [ctx - 777 * b for b in range(seqs)] + [3, 64]
    attend_and_check(Batch(lens, [1] * len(lens), 1, 128, 64, kind, ctx), 4, x, workspace=workspace)


def test_attention_repeats_bit_for_bit():
    """The order of the parts does not depend on timing, and a workspace can be used again."""
    bt = Batch([7000, 1, 350, 2500], [1, 1, 2, 1], 2, 128, 16, "int8", 8)
    out, lse, q, ws = attend_and_check(bt, 8, "f32")
    for _ in range(5):
        l2 = torch.empty_like(lse)
        o2 = om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, 2, lse=l2, workspace=ws)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_attention_rows_that_see_nothing():
    """No context at all, and more queries than tokens: zeros and -inf."""
    attend_and_check(Batch([0, 2, 0, 40], [1, 4, 3, 1], 1, 64, 16, "int8", 2), 2, "f32")


def test_attention_without_tokens_for_a_sequence():
    attend_and_check(Batch([50, 20, 30], [0, 2, 0], 2, 64, 16, "e4m3", 2), 4, "f16")


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_attention_ignores_what_the_mask_hides(x):
    """Stale codes (NaN among them) behind the end, NaN scales of pages outside the window or past the end."""
    ctx, new = [70, 37, 100], [1, 2, 1]
    bt = Batch(ctx, new, 2, 128, 16, "e4m3", 21)
    for b, c in enumerate(ctx):
        pid, row = bt.table_np[b][(c - 1) // 16], (c - 1) % 16
        for t in (bt.k, bt.v):
            t.view(torch.int8)[pid, :, row + 1:] = 0x7F
        for j in range((c - new[b] - 20 + 1) // 16):
            bt.ks[bt.table_np[b][j]] = float("nan")
            bt.vs[bt.table_np[b][j]] = float("inf")
            bt.k.view(torch.int8)[bt.table_np[b][j]] = 0x7F
    bt.ks[torch.from_numpy(bt.spare).cuda()] = float("nan")
    bt.table_np[:, -1] = bt.spare[0]
    attend_and_check(bt, 4, x, window=20)


def test_attention_shows_a_page_that_is_not_finite():
    bt = Batch([64, 64], [1, 1], 1, 64, 16, "int8", 5).device()
    bt.vs[int(bt.table_np[0][1])] = float("nan")
    q = torch.randn(2, 2, 64, device="cuda")
    out = om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, 1)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()
    bt.vs[int(bt.table_np[0][1])] = 1.0
    bt.ks[int(bt.table_np[0][2])] = float("nan")
    out = om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, 1)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


def test_attention_table_entries_outside_the_cache_are_not_followed():
    bt = Batch([100, 60], [1, 2], 2, 128, 16, "int8", 6, width_extra=0)
    bt.table_np[0, 2], bt.table_np[1, 0] = -1, bt.pages
    bt.table_np[0, 5] = 2 ** 31 - 1
    attend_and_check(bt, 4, "f32")
    bt = Batch([100, 60], [1, 2], 2, 128, 16, "int8", 6, width_extra=0)
    bt.table_np = bt.table_np[:, :3]  # positions behind the table
    attend_and_check(bt, 4, "bf16")


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
def test_attention_wide_ranges(x):
    """Large scores, values of very different scale by page, zero scales, queries of very different size."""
    bt = Batch([300, 300, 300], [1, 1, 1], 1, 128, 16, "int8", 31)
    scales = 10.0 ** torch.linspace(-4, 2, bt.pages, device="cuda")
    bt.vs = scales[torch.randperm(bt.pages, generator=gen(1), device="cuda")][:, None].contiguous()
    bt.vs[int(bt.table_np[0][0])] = 0.0
    bt.ks[int(bt.table_np[1][3])] = 0.0
    q = torch.randn(3, 4, 128, generator=gen(2), device="cuda")
    q[0] *= 30.0
    q[1] *= 1e-3
    q[2, 0] = 0.0
    q[2, 1] *= 1e4 if x == "f16" else 1e6
    if x != "f16":
        q[2, 2] *= 1e-30
    attend_and_check(bt, 4, x, q=q.to(ref.TORCH[x]), scale=0.01)


def test_attention_strided_queries_and_outputs():
    bt = Batch([40, 90], [2, 1], 2, 64, 32, "int8", 3).device()
    rows = torch.randn(3, 12, 64, generator=gen(4), device="cuda").bfloat16()
    q = rows[:, 2:10]
    outs = torch.full((3, 20, 64), 7.0, device="cuda").bfloat16()
    ws = om.new_kv_workspace(bt.cache, 8, 2)
    om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, 2, out=outs[:, 1:17:2], workspace=ws)
    want = om.kv_attention(bt.cache, q.contiguous(), bt.table, bt.lens, bt.cu, 2, workspace=ws)
    assert torch.equal(outs[:, 1:17:2], want)
    assert (outs[:, 0::2] == 7).all() and (outs[:, 17:] == 7).all()


def test_attention_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: pages at its far end."""
    free, _ = torch.cuda.mem_get_info()
    if free < 30 << 30:
        pytest.skip("less than 30 GB of device memory free")
    page, hkv, dim = 128, 8, 128
    pages = (1 << 32) // (page * hkv * dim) + 40
    k = torch.zeros(pages, hkv, page, dim, dtype=torch.int8, device="cuda")
    v = torch.zeros(pages, hkv, page, dim, dtype=torch.int8, device="cuda")
    ks, vs = torch.zeros(pages, hkv, device="cuda"), torch.zeros(pages, hkv, device="cuda")
    small = Batch([700], [1], hkv, dim, page, "int8", 12, width_extra=0, shuffle=False).device()
    n = small.pages
    k[-n:], v[-n:], ks[-n:], vs[-n:] = small.k, small.v, small.ks, small.vs
    big = om.PagedKVCache(k, v, ks, vs)
    q = torch.randn(1, 16, dim, generator=gen(1), device="cuda")
    ws = om.new_kv_workspace(big, 16, 1)
    far = small.table + (pages - n)
    a = om.kv_attention(big, q, far.int(), small.lens, small.cu, 1, workspace=ws)
    b = om.kv_attention(small.cache, q, small.table, small.lens, small.cu, 1, workspace=ws)
    assert torch.equal(a, b)
    new = torch.randn(1, hkv, dim, generator=gen(2), device="cuda")
    for c, t in ((big, far.int()), (small.cache, small.table)):
        om.kv_append(c, None, new, new, None, t, small.lens, small.cu, 1)
    cu = i32([0, 700])
    got = [om.kv_read(c, t, i32([0]), cu, 700, 700) for c, t in ((big, far.int()), (small.cache, small.table))]
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert (k[0] == 0).all() and (k[(pages - n) // 2] == 0).all()
    del k, v, big
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ append
def bits(a):
    return np.ascontiguousarray(a, np.float32).view(np.uint32)


def append_and_check(bt, hq, x, rot, pairs, seed=0, mutate=None, in_place=False, rows=None):
    bt.device()
    T = int(bt.cu_np[-1])
    fused = torch.randn(T, hq + 2 * bt.hkv, bt.dim, generator=gen(seed), device="cuda").to(ref.TORCH[x])
    if mutate:
        mutate(fused)
    q, k, v = fused[:, :hq], fused[:, hq:hq + bt.hkv], fused[:, hq + bt.hkv:]
    rows = max(max(bt.ctx), 1) if rows is None else rows
    table = om.rope_table(rows, rot, base=1000.0) if rot else None
    pos = np.concatenate([np.arange(c - n, c) for c, n in zip(bt.ctx, bt.new)]) if T else np.zeros(0, int)
    as32 = lambda t: t.float().cpu().numpy()
    tab = table.cpu().numpy() if rot else np.zeros((0, 0, 2), np.float32)
    want_q = torch.from_numpy(ref.rotate(as32(q), tab, pos, rot, pairs == "interleaved")).to(q.dtype)
    want = []
    for codes, scales, new in ((bt.k, bt.ks, ref.rotate(as32(k), tab, pos, rot, pairs == "interleaved")), (bt.v, bt.vs, as32(v))):
        want.append(ref.append(codes.view(torch.int8).cpu().numpy(), scales.cpu().numpy(), new, bt.table_np, bt.ctx, bt.cu_np, bt.page, bt.kind))
    got = om.kv_append(bt.cache, q, k, v, table, bt.table, bt.lens, bt.cu, max(max(bt.new), 1), pairs=pairs, q_out=q if in_place else None)
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
    return fused, table


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot,page", [(64, 64, 16), (128, 128, 32), (128, 64, 64), (256, 24, 16), (128, 0, 128)])
def test_append_bit_for_bit(dim, rot, page, pairs, x, kind):
    ctx, new = [1, 17, 16, 40, 200, 33], [1, 1, 1, 3, 70, 33]
    append_and_check(Batch(ctx, new, 2, dim, page, kind, dim + rot), 6, x, rot, pairs)


def test_append_in_place_and_without_queries():
    append_and_check(Batch([9, 50], [2, 50], 3, 64, 16, "int8", 1), 3, "bf16", 64, "half", in_place=True)
    append_and_check(Batch([9, 50], [2, 50], 3, 64, 16, "int8", 1), 3, "f32", 32, "interleaved", in_place=True)
    bt = Batch([9, 50], [1, 4], 2, 128, 16, "e4m3", 1).device()
    k = torch.randn(5, 2, 128, generator=gen(0), device="cuda")
    assert om.kv_append(bt.cache, None, k, k, None, bt.table, bt.lens, bt.cu, 4) is None


def test_append_values_that_are_not_finite_show():
    def mutate(f):
        f[0, 2, 5] = float("nan")    # a key of sequence 0
        f[1, 4, 7] = float("inf")    # a value of sequence 1
        f[2, 3] = 0.0                # a head of zeros
    append_and_check(Batch([20, 1, 33], [1, 1, 1], 2, 64, 16, "int8", 1), 2, "f32", 64, "half", mutate=mutate)
    append_and_check(Batch([20, 1, 33], [1, 1, 1], 2, 64, 16, "e4m3", 1), 2, "f32", 64, "half", mutate=mutate)


def test_append_extreme_magnitudes():
    def mutate(f):
        f[0] *= 1e30
        f[1] *= 1e-42
        f[2] *= 1e-38
    for kind in ("int8", "e4m3"):
        append_and_check(Batch([20, 1, 33], [1, 1, 1], 2, 64, 16, kind, 1), 2, "f32", 0, "half", mutate=mutate)


def test_append_positions_outside_table_and_cache():
    """Positions behind the rotation table turn to NaN; pages outside the cache are not written."""
    append_and_check(Batch([40, 12], [3, 2], 2, 64, 16, "int8", 7), 2, "f32", 64, "half", rows=38)
    bt = Batch([40, 12, 50], [20, 2, 30], 2, 64, 16, "int8", 7, width_extra=0)
    bt.table_np[0, 1], bt.table_np[1, 0], bt.table_np[2, 2] = -5, bt.pages, 2 ** 31 - 1
    append_and_check(bt, 2, "bf16", 32, "half")
    bt = Batch([40, 12], [3, 2], 2, 64, 16, "int8", 7)
    bt.table_np = bt.table_np[:, :2]
    append_and_check(bt, 2, "f32", 0, "half")


def test_append_more_new_tokens_than_context():
    """Tokens at negative positions are not stored; their queries are NaN under a rotation."""
    append_and_check(Batch([2, 0, 20], [4, 3, 1], 1, 64, 16, "int8", 7), 2, "f32", 64, "half")


def test_append_unaligned_operands():
    bt = Batch([20, 31], [2, 1], 2, 64, 16, "int8", 5)
    keep = (bt.k.clone(), bt.v.clone(), bt.ks.clone(), bt.vs.clone())
    fused, table = append_and_check(bt, 2, "bf16", 64, "half", seed=3)
    other = om.PagedKVCache(*keep)
    wide = torch.zeros(3, 6 * 64 + 7, dtype=fused.dtype, device="cuda")
    odd = torch.as_strided(wide, fused.shape, (6 * 64 + 7, 64, 1), 1)
    odd.copy_(fused)
    outs = torch.as_strided(torch.zeros(3 * 200 + 3, dtype=fused.dtype, device="cuda"), (3, 2, 64), (200, 65, 1), 3)
    q = om.kv_append(other, odd[:, :2], odd[:, 2:4], odd[:, 4:], table, bt.table, bt.lens, bt.cu, 2, q_out=outs)
    assert torch.equal(other.k, bt.k) and torch.equal(other.v, bt.v) and torch.equal(other.k_scale, bt.ks)
    want = om.kv_append(other, fused[:, :2], fused[:, 2:4], fused[:, 4:], table, bt.table, bt.lens, bt.cu, 2)
    assert torch.equal(q, want)


def test_append_one_token_at_a_time_reads_back():
    """A sequence built token by token: each value within half a unit of the scale for each time
    its page's scale grew."""
    page, dim, n = 16, 64, 40
    cache = om.PagedKVCache.empty(4, 1, page, dim)
    table, cu = i32([[2, 0, 3]]), i32([0, 1])
    x = torch.randn(n, 1, dim, generator=gen(5), device="cuda")
    growths = np.zeros(4)
    for t in range(n):
        before = cache.v_scale[:, 0].cpu().numpy().copy()
        om.kv_append(cache, None, x[t:t + 1], x[t:t + 1], None, table, i32([t + 1]), cu, 1)
        growths += cache.v_scale[:, 0].cpu().numpy() != before
    k, v = om.kv_read(cache, table, i32([0]), i32([0, n]), n, n)
    assert torch.equal(k, v)
    for j, pid in enumerate((2, 0, 3)):
        part = slice(j * page, min(n, (j + 1) * page))
        s = float(cache.v_scale[pid, 0])
        assert s >= float(x[part].abs().max()) / 127 * (1 - 1e-6)
        assert float((v[part] - x[part]).abs().max()) <= growths[pid] * 0.5 * s * (1 + 1e-5) + 1e-6


# -------------------------------------------------------------- read, table
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("page,dim", [(16, 64), (64, 128), (32, 256)])
def test_read_back_bit_for_bit(page, dim, x, kind):
    ctx, new = [1, 100, 33, 16, 0], [1, 77, 20, 16, 0]
    bt = Batch(ctx, new, 3, dim, page, kind, 9).device()
    T = sum(new)
    start = [c - n for c, n in zip(ctx, new)]
    k, v = om.kv_read(bt.cache, bt.table, i32(start), bt.cu, max(new), T, dtype=ref.TORCH[x])
    for got, codes, scales in ((k, bt.k, bt.ks), (v, bt.v, bt.vs)):
        c, s = ref.code_values(codes).astype(np.float32), scales.cpu().numpy()
        rows = []
        for b in range(len(ctx)):
            pos = np.arange(start[b], ctx[b])
            ids = bt.table_np[b][pos // page]
            rows.append(c[ids, :, pos % page] * s[ids][:, :, None])
        want = torch.from_numpy(np.concatenate(rows)).to(ref.TORCH[x])
        assert torch.equal(got.cpu(), want)


def test_read_positions_the_cache_does_not_hold():
    bt = Batch([40], [40], 1, 64, 16, "int8", 9, width_extra=0)
    bt.table_np[0, 1] = -1
    bt.device()
    k, v = om.kv_read(bt.cache, bt.table, i32([-2]), i32([0, 60]), 60, 60)
    nan = torch.isnan(k[:, 0, 0]).cpu().numpy()
    pos = np.arange(-2, 58)
    assert (nan == ((pos < 0) | (pos // 16 == 1) | (pos >= 48))).all()
    assert (torch.isnan(v).all(-1).all(-1).cpu().numpy() == nan).all()


@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0)])
@pytest.mark.parametrize("rot", [2, 64, 128])
def test_rope_table(scaling, factor, rot):
    rows, base, original = 5000, 10000.0, 1024
    t = om.rope_table(rows, rot, base=base, scaling=scaling, factor=factor, original=original).cpu().numpy()
    i = np.arange(rot // 2)
    b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" and rot > 2 else base
    f, amp = b ** (-2.0 * i / rot), 1.0
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        where = lambda beta: rot * np.log(original / (beta * 2 * np.pi)) / (2 * np.log(base))
        lo, hi = max(np.floor(where(32.0)), 0), min(np.ceil(where(1.0)), rot - 1)
        hi = hi + 0.001 if lo == hi else hi
        ramp = np.clip((i - lo) / (hi - lo), 0, 1)
        f, amp = f / factor * ramp + f * (1 - ramp), 0.1 * np.log(factor) + 1
    a = np.arange(rows)[:, None] * f
    # a 64-bit angle of up to 5000, then one rounding to 32 bits
    tol = 2.0 ** -24 * amp + 1e-11
    assert np.abs(t[..., 0] - amp * np.cos(a)).max() <= tol and np.abs(t[..., 1] - amp * np.sin(a)).max() <= tol
