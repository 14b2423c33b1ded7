"""Measured cases of the decoding operators: the 4-bit matrix-vector product,
appending rotated keys and values to a paged 8-bit cache, attention over that
cache, and reading the cache back as values.

``run`` computes an operator either by the library's entry points
(``own = True``) or by its plain form in elementary torch operations
(``own = False``); ``exact`` computes the definition in 64 bits.

Definitions
-----------
4-bit product: y[i][j] = sum_p x[i][p] * (u[j][p] - z[j][p / group]) * s[j][p / group], with u the
unsigned 4-bit code (the low half of byte p / 2 for even p), z = 8 where no zeros are given.

Cache: codes [pages][kv heads][page][head dim], one 32-bit scale for each page and head; a value is
code * scale. Sequence b's token at position t lies in page block_table[b][t / page], row t % page.

Append: the new tokens of sequence b are its last ones, at positions ctx_len[b] - new ...
ctx_len[b] - 1. Queries and keys are rotated by their position's row of a (cos, sin) table:
(a, b) -> (a c - b s, b c + a s) for the pairs of the first rot elements, each product and sum rounded
to 32 bits. A page's scale is the larger of its old one (none, if its first row is new) and
fl(largest new magnitude * fl(1 / top)), top = 127 (int8) or 448 (e4m3); old codes of a page whose
scale grew become round(code * (old / new)), new codes are round(value / scale).

Attention: query i of sequence b (at position p = ctx_len[b] - queries + i) attends to the
positions max(0, p - window + 1) .. p (window 0: all from 0). Outputs are the softmax-weighted
values and the natural log of the sum of exponentials.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BITS = {"f32": 4, "f16": 2, "bf16": 2}
TOP = {"int8": 127.0, "e4m3": 448.0}


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # One token through a small projection: the call's latency.
        {"name": "w4 one token small", "op": "w4", "m": 1, "n": 1024, "k": 1024, "group": 128, "zeros": False, "x": "f16"},
        # The library's decode product (1 x 11008 x 4096) with 4-bit weights, 32-bit activations.
        {"name": "w4 decode f32", "op": "w4", "m": 1, "n": 11008, "k": 4096, "group": 128, "zeros": False, "x": "f32"},
        # A batch of 16 sequences through a wide projection, small groups with zero points, ragged
        # sizes (rows that are not 16-byte aligned), about 130 MB of weights.
        {"name": "w4 batch wide", "op": "w4", "m": 16, "n": 28669, "k": 8178, "group": 32, "zeros": True, "x": "bf16"},
        # One token for each of 4 sequences: the call's latency.
        {"name": "append 4 tokens", "op": "append", "seqs": 4, "new": 1, "ctx": 700, "hq": 32, "hkv": 8, "dim": 128, "page": 16, "kv": "int8", "x": "bf16", "rot": 128, "pairs": "half"},
        # One token for each of 192 sequences, part of the head rotated, neighbouring pairs.
        {"name": "append batch 192", "op": "append", "seqs": 192, "new": 1, "ctx": 4000, "hq": 32, "hkv": 8, "dim": 128, "page": 64, "kv": "e4m3", "x": "f16", "rot": 64, "pairs": "interleaved"},
        # Prompts of up to 4096 tokens for 4 sequences that have some tokens already.
        {"name": "append prompts", "op": "append", "seqs": 4, "new": 4096, "ctx": 5001, "hq": 32, "hkv": 8, "dim": 128, "page": 32, "kv": "int8", "x": "f32", "rot": 128, "pairs": "half"},
        # One short sequence: the call's latency.
        {"name": "attend one short", "op": "attend", "seqs": 1, "q": 1, "ctx": 331, "hq": 16, "hkv": 4, "dim": 64, "page": 16, "window": 0, "kv": "int8", "x": "bf16"},
        # One long sequence: the cache split over the whole GPU.
        {"name": "attend one long", "op": "attend", "seqs": 1, "q": 1, "ctx": 131071, "hq": 32, "hkv": 8, "dim": 128, "page": 16, "window": 0, "kv": "e4m3", "x": "f16"},
        # 64 sequences of up to 16K tokens, 8 query heads to a key head: about 1.1 GB of cache.
        {"name": "attend batch 64", "op": "attend", "seqs": 64, "q": 1, "ctx": 16384, "hq": 64, "hkv": 8, "dim": 128, "page": 64, "window": 0, "kv": "int8", "x": "bf16"},
        # Checking up to 5 drafted tokens of 24 sequences at once, 32-bit, sliding window.
        {"name": "attend drafts f32", "op": "attend", "seqs": 24, "q": 5, "ctx": 9000, "hq": 30, "hkv": 6, "dim": 128, "page": 32, "window": 4096, "kv": "int8", "x": "f32"},
        # One page-sized piece read back.
        {"name": "read 40 tokens", "op": "read", "seqs": 1, "len": 40, "ctx": 300, "hkv": 8, "dim": 128, "page": 16, "kv": "int8", "x": "f32"},
        # Whole prompts read back, as for a product over them in 16 bits.
        {"name": "read prompts", "op": "read", "seqs": 8, "len": 12000, "ctx": 12345, "hkv": 8, "dim": 128, "page": 64, "kv": "e4m3", "x": "bf16"},
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v + (v == 3 << 10)


def draw(rng):
    op = rng.choice(("w4", "append", "attend", "attend", "read", "w4"))
    x = rng.choice(("f32", "f16", "bf16"))
    kv = rng.choice(("int8", "e4m3"))
    if op == "w4":
        group = rng.choice((32, 64, 128))
        k = _log(rng, 512, 12288)
        n = min(_log(rng, 512, 32768), (28669 * 8178) // k)
        return {"op": op, "m": _log(rng, 1, 16), "n": n, "k": k, "group": group, "zeros": rng.random() < 0.5, "x": x}
    dim, page = rng.choice((64, 128, 128, 256)), rng.choice((16, 32, 64, 128))
    hkv = rng.choice((1, 2, 4, 5, 8))
    if op == "append":
        seqs = _log(rng, 1, 192)
        new = 1 if rng.random() < 0.5 else max(1, _log(rng, 1, 4096) // seqs)
        hq = hkv * rng.choice((2, 5, 8))
        return {"op": op, "seqs": seqs, "new": new, "ctx": new + _log(rng, 1, 4000), "hq": hq, "hkv": hkv, "dim": dim, "page": page, "kv": kv, "x": x,
                "rot": rng.choice((dim, dim, dim // 2)), "pairs": rng.choice(("half", "interleaved"))}
    if op == "read":
        seqs = _log(rng, 1, 16)
        length = max(1, min(_log(rng, 16, 12000), 96000 * 1024 // (seqs * hkv * dim)))
        return {"op": op, "seqs": seqs, "len": length, "ctx": length + _log(rng, 1, 500), "hkv": hkv, "dim": dim, "page": page, "kv": kv, "x": x}
    seqs = _log(rng, 1, 64)
    group = rng.choice((1, 2, 4, 5, 8))
    q = rng.choice((1, 1, 1, 2, 4, 8))
    ctx = min(_log(rng, 100, 131072), 64 * 16384 * 1024 // (seqs * hkv * dim * max(1, q * group // 8)))
    return {"op": op, "seqs": seqs, "q": q, "ctx": max(ctx, 8), "hq": hkv * group, "hkv": hkv, "dim": dim, "page": page,
            "window": rng.choice((0, 0, 1024)), "kv": kv, "x": x}


# ------------------------------------------------------ lengths, by the case
def _share(b):
    """0.5 .. 1, spread evenly over the sequences, the first one 1."""
    return 1.0 - 0.5 * ((b * 0.6180339887498949) % 1.0)


def _lengths(case):
    """(ctx, new) of each sequence; new: the tokens appended, queried or read."""
    ctx = [max(1, int(case["ctx"] * _share(b))) for b in range(case["seqs"])]
    if case["op"] == "append":
        new = [max(1, int(case["new"] * _share(3 * b))) for b in range(case["seqs"])]
        ctx = [max(c, t) for c, t in zip(ctx, new)]
    elif case["op"] == "attend":
        new = [max(1, int(case["q"] * _share(3 * b))) for b in range(case["seqs"])]
    else:
        new = [max(1, int(case["len"] * _share(b))) for b in range(case["seqs"])]
        ctx = [max(c, t) for c, t in zip(ctx, new)]
    return ctx, new


def _append_reads(case):
    """First position and count, for each sequence, of the tokens in the pages that an append touches."""
    ctx, new = _lengths(case)
    first = [(c - t) // case["page"] * case["page"] for c, t in zip(ctx, new)]
    return first, [c - f for c, f in zip(ctx, first)]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(counts):
    return _i32([0] + list(np.cumsum(counts)))


def _cu_host(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


# --------------------------------------------------------------- the inputs
def _rotation_table(rows, rot):
    """cos and sin of position * 10000^(-2 i / rot), from 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.stack((angle.cos(), angle.sin()), -1).float().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = {"generator": g, "device": "cuda"}
    s = {"case": case}
    if case["op"] == "w4":
        m, n, k = case["m"], case["n"], case["k"]
        groups = -(-k // case["group"])
        s["x"] = torch.randn(m, k, **kw).to(DTYPES[case["x"]])
        s["u"] = torch.randint(0, 256, (n, (k + 1) // 2), dtype=torch.uint8, **kw)
        s["s"] = (0.02 * (0.5 + torch.rand(n, groups, **kw)) / 4).to(torch.float32 if case["x"] == "f32" else DTYPES[case["x"]])
        s["z"] = torch.randint(4, 12, (n, groups), dtype=torch.uint8, **kw) if case["zeros"] else None
        return s
    seqs, hkv, dim, page = case["seqs"], case["hkv"], case["dim"], case["page"]
    ctx, new = _lengths(case)
    width = -(-max(ctx) // page)
    pages = sum(-(-c // page) for c in ctx) + 3
    order = torch.randperm(pages, **kw).to(torch.int32)
    # every sequence its own pages, in random order; unused places of the table hold page 0
    table = torch.zeros(seqs, width, dtype=torch.int32, device="cuda")
    used = [-(-c // page) for c in ctx]
    live = torch.arange(width, device="cuda")[None, :] < _i32(used)[:, None]
    table[live] = order[: sum(used)]
    codes = []
    for _ in range(2):  # keys, values
        if case["kv"] == "int8":
            c = torch.randn(pages, hkv, page, dim, dtype=torch.float16, **kw).mul_(38).clamp_(-127, 127).round_().to(torch.int8)
        else:
            c = torch.randn(pages, hkv, page, dim, dtype=torch.float16, **kw).mul_(110).clamp_(-448, 448).to(torch.float8_e4m3fn)
        codes.append(c)
    top = TOP[case["kv"]]
    s["k"], s["v"] = codes
    s["ks"], s["vs"] = (((0.7 + 0.6 * torch.rand(pages, hkv, **kw)) * (3.3 / top)).contiguous() for _ in range(2))
    s["table"], s["ctx"] = table, _i32(ctx)
    s["cu"], s["total"], s["most"] = _cu(new), sum(new), max(new)
    if case["op"] == "read":
        s["first"] = _i32([c - t for c, t in zip(ctx, new)])
    else:
        heads = case["hq"] + (2 * hkv if case["op"] == "append" else 0)
        # queries (keys and values) are parts of one product's output rows
        rows = torch.randn(sum(new), heads, dim, **kw)
        if case["op"] == "attend":
            rows *= 1.5
        rows = rows.to(DTYPES[case["x"]])
        s["q"] = rows[:, : case["hq"]]
        if case["op"] == "append":
            s["knew"], s["vnew"] = rows[:, case["hq"]: case["hq"] + hkv], rows[:, case["hq"] + hkv:]
            s["rot"] = _rotation_table(max(ctx) + 1, case["rot"])
            first, count = _append_reads(case)
            s["first"], s["rcu"], s["rmost"], s["rtotal"] = _i32(first), _cu(count), max(count), sum(count)
    if own:
        import implicit_gemm_convolution_gb300 as om
        s["cache"] = om.PagedKVCache(s["k"], s["v"], s["ks"], s["vs"])
        if case["op"] == "attend":
            s["ws"] = om.new_kv_workspace(s["cache"], case["hq"], s["most"])
            s["lse"] = torch.empty(s["total"], case["hq"], dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import implicit_gemm_convolution_gb300 as om
    case = s["case"]
    if case["op"] == "w4":
        return om.w4_matvec(s["x"], s["u"], s["s"], zeros=s["z"], group=case["group"])
    if case["op"] == "append":
        q = om.kv_append(s["cache"], s["q"], s["knew"], s["vnew"], s["rot"], s["table"], s["ctx"], s["cu"], s["most"], pairs=case["pairs"])
        # the cache as the values it stands for
        k, v = om.kv_read(s["cache"], s["table"], s["first"], s["rcu"], s["rmost"], s["rtotal"])
        return q, k, v, s["ks"], s["vs"]
    if case["op"] == "attend":
        out = om.kv_attention(s["cache"], s["q"], s["table"], s["ctx"], s["cu"], s["most"], window=case["window"], lse=s["lse"], workspace=s["ws"])
        return out, s["lse"]
    return om.kv_read(s["cache"], s["table"], s["first"], s["cu"], s["most"], s["total"], dtype=DTYPES[case["x"]])


def _run_plain(s):
    return {"w4": _plain_w4, "append": _plain_append, "attend": _plain_attend, "read": _plain_read}[s["case"]["op"]](s)


def _plain_w4(s):
    case = s["case"]
    n, k, group = case["n"], case["k"], case["group"]
    u = torch.stack((s["u"] & 15, s["u"] >> 4), -1).reshape(n, -1)[:, :k].float()
    z = s["z"].float().repeat_interleave(group, 1)[:, :k] if s["z"] is not None else 8.0
    w = (u - z) * s["s"].float().repeat_interleave(group, 1)[:, :k]
    return (s["x"].float() @ w.t()).to(s["x"].dtype)


def _tokens(s, first, cu, total):
    """Sequence and position of each of `total` tokens, `first` the position of a sequence's first."""
    i = torch.arange(total, device="cuda")
    b = torch.searchsorted(cu[1:].long(), i, right=True)
    return b, first.long()[b] + (i - cu.long()[b])


def _rotate(x, cs, rot, pairs):
    x = x.float()
    c, d = cs[:, None, :, 0], cs[:, None, :, 1]
    if pairs == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        return torch.cat((a * c - b * d, b * c + a * d, x[..., rot:]), -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat((torch.stack((a * c - b * d, b * c + a * d), -1).flatten(-2), x[..., rot:]), -1)


def _to_codes(x, scale, kind):
    x = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0)
    return _round_codes(x, kind)


def _round_codes(x, kind):
    x = x.clamp(-TOP[kind], TOP[kind])
    return x.round().to(torch.int8) if kind == "int8" else x.to(torch.float8_e4m3fn)


def _plain_append(s):
    case = s["case"]
    page, kind, hkv = case["page"], case["kv"], case["hkv"]
    counts = s["cu"][1:] - s["cu"][:-1]
    b, pos = _tokens(s, s["ctx"] - counts, s["cu"], s["total"])
    cs = s["rot"][pos]
    q = _rotate(s["q"], cs, case["rot"], case["pairs"]).to(s["q"].dtype)
    at, row = s["table"].long()[b, pos // page], pos % page
    heads = torch.arange(hkv, device="cuda")
    # only a sequence's first page can have rows that are kept
    start = (s["ctx"] - counts).long()
    head_page = s["table"].long()[torch.arange(case["seqs"], device="cuda"), start // page]
    had = (start % page > 0)[:, None]
    for codes, scales, new in ((s["k"], s["ks"], _rotate(s["knew"], cs, case["rot"], case["pairs"])), (s["v"], s["vs"], s["vnew"].float())):
        old = torch.zeros_like(scales).index_copy_(0, head_page, torch.where(had, scales[head_page], 0.0))
        top = torch.zeros_like(scales).index_reduce_(0, at, new.abs().amax(-1), "amax", include_self=True)
        grown = torch.maximum(old, top * (1.0 / TOP[kind]))
        ratio = torch.where(grown > 0, old / torch.where(grown > 0, grown, 1.0), 0.0)[head_page]
        raw = codes.view(torch.int8)
        was = raw[head_page].view(codes.dtype).float()
        raw.index_copy_(0, head_page, _round_codes(was * ratio[:, :, None, None], kind).view(torch.int8))
        scales.index_copy_(0, at, grown[at])
        raw[at[:, None], heads, row[:, None]] = _to_codes(new, grown[at][:, :, None], kind).view(torch.int8)
    k, v = _values(s, *_tokens(s, s["first"], s["rcu"], s["rtotal"]), torch.float32)
    return q, k, v, s["ks"], s["vs"]


def _values(s, b, pos, dtype):
    page = s["case"]["page"]
    at, row, heads = s["table"].long()[b, pos // page], pos % page, torch.arange(s["case"]["hkv"], device="cuda")

    def part(codes, scales):
        c = codes.view(torch.int8)[at[:, None], heads, row[:, None]].view(codes.dtype)
        return (c.float() * scales[at][:, :, None]).to(dtype)

    return part(s["k"], s["ks"]), part(s["v"], s["vs"])


def _plain_read(s):
    return _values(s, *_tokens(s, s["first"], s["cu"], s["total"]), DTYPES[s["case"]["x"]])


def _plain_attend(s):
    case = s["case"]
    seqs, hq, hkv, dim, most = case["seqs"], case["hq"], case["hkv"], case["dim"], s["most"]
    counts = s["cu"][1:] - s["cu"][:-1]
    b, pos = _tokens(s, s["ctx"] - counts, s["cu"], s["total"])
    i = torch.arange(s["total"], device="cuda") - s["cu"].long()[b]
    q = torch.zeros(seqs, most, hq, dim, device="cuda").index_put_((b, i), s["q"].float())
    p = torch.full((seqs, most), -1, device="cuda").index_put_((b, i), pos)
    table = s["table"].long()

    def whole(codes, scales):  # seqs x heads x positions x dim
        c = codes.view(torch.int8)[table].view(codes.dtype).float().mul_(scales[table][..., None, None])
        return c.transpose(1, 2).reshape(seqs, hkv, -1, dim)

    q = q.transpose(1, 2).reshape(seqs, hkv, (hq // hkv) * most, dim)  # heads of a group, then queries
    scores = (q @ whole(s["k"], s["ks"]).transpose(2, 3)).mul_(dim ** -0.5)
    scores = scores.view(seqs, hq, most, -1)
    t = torch.arange(scores.shape[-1], device="cuda")
    seen = t <= p[..., None]
    if case["window"]:
        seen &= t > p[..., None] - case["window"]
    scores.masked_fill_(~seen[:, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    e = scores.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    out = (e.view(seqs, hkv, -1, e.shape[-1]) @ whole(s["v"], s["vs"])).view(seqs, hq, most, dim) / total.clamp(min=1e-38)
    lse = (total.log() + top)[..., 0]
    return out.transpose(1, 2)[b, i].to(s["q"].dtype), lse.transpose(1, 2)[b, i]


# ---------------------------------------------------------- the bare work
def work(case):
    x = BITS[case["x"]]
    if case["op"] == "w4":
        m, n, k = case["m"], case["n"], case["k"]
        groups = -(-k // case["group"])
        return {"bytes": m * k * x + n * ((k + 1) // 2) + n * groups * (x + bool(case["zeros"])) + m * n * x, "flops": 2 * m * n * k}
    ctx, new = _lengths(case)
    hkv, dim, page = case["hkv"], case["dim"], case["page"]
    if case["op"] == "attend":
        hq, w = case["hq"], case["window"]
        pairs = sum(min(c - t + i + 1, w or c) for c, t in zip(ctx, new) for i in range(t))
        rows = [min(c, w + t - 1) if w else c for c, t in zip(ctx, new)]
        spots = sum(-(-r // page) for r in rows)
        return {"bytes": sum(rows) * hkv * dim * 2 + spots * (hkv * 8 + 4) + sum(new) * hq * (2 * dim * x + 4), "flops": 4 * pairs * hq * dim}
    if case["op"] == "read":
        return {"bytes": sum(new) * hkv * dim * 2 * (1 + x), "flops": sum(new) * hkv * dim * 2}
    first, count = _append_reads(case)
    old = sum(count) - sum(new)
    one = sum(new) * dim
    rewritten = 2 * hkv * dim * 2 * old  # the codes of a page whose scale grows, once in and once out
    values = sum(count) * hkv * dim * 2 * (1 + 4)
    return {"bytes": one * (2 * case["hq"] + 2 * hkv) * x + one * hkv * 2 + sum(new) * case["rot"] * 4 + rewritten + values,
            "flops": one * (case["hq"] + hkv) * 3 + one * hkv * 4}


# --------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    global own
    kept, own = own, False
    s = prepare(case, seed)
    own = kept
    return {"w4": _exact_w4, "append": _exact_append, "attend": _exact_attend, "read": _exact_read}[case["op"]](s)


def _exact_w4(s):
    case = s["case"]
    n, k, group = case["n"], case["k"], case["group"]
    x, y = s["x"].double(), []
    step = max(1, (1 << 26) // k)
    for j in range(0, n, step):
        raw = s["u"][j: j + step].to(torch.int64)
        codes = torch.empty(raw.shape[0], 2 * raw.shape[1], dtype=torch.float64, device="cuda")
        codes[:, 0::2], codes[:, 1::2] = raw % 16, raw // 16
        at = torch.arange(k, device="cuda") // group
        zero = s["z"][j: j + step].double()[:, at] if case["zeros"] else torch.tensor(8.0, dtype=torch.float64, device="cuda")
        y.append(x @ ((codes[:, :k] - zero) * s["s"][j: j + step].double()[:, at]).t())
    return torch.cat(y, 1)


def _sequence(s, b, lo, hi):
    """Keys and values of positions lo .. hi - 1 of sequence b: heads x positions x dim."""
    page = s["case"]["page"]
    first, last = lo // page, -(-hi // page)
    ids = s["table"][b, first:last].long()
    out = []
    for codes, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        c = codes.view(torch.int8)[ids].view(codes.dtype).to(torch.float32).double() * scales[ids].double()[:, :, None, None]
        out.append(c.transpose(0, 1).flatten(1, 2)[:, lo - first * page: hi - first * page])
    return out


def _exact_read(s):
    ctx, new = _lengths(s["case"])
    got = [_sequence(s, b, c - t, c) for b, (c, t) in enumerate(zip(ctx, new))]
    return tuple(torch.cat([g[j].transpose(0, 1) for g in got]) for j in range(2))


def _exact_attend(s):
    case = s["case"]
    ctx, new = _lengths(case)
    at, group = _cu_host(new), case["hq"] // case["hkv"]
    outs, sums = [], []
    for b, (c, t) in enumerate(zip(ctx, new)):
        lo = max(0, c - t - case["window"] + 1) if case["window"] else 0
        k, v = _sequence(s, b, lo, c)
        q = s["q"][at[b]: at[b + 1]].double()
        here = torch.arange(c - t, c, device="cuda")[:, None]
        there = torch.arange(lo, c, device="cuda")[None, :]
        hidden = there > here
        if case["window"]:
            hidden |= there <= here - case["window"]
        rows, logs = [], []
        for h in range(case["hkv"]):
            w = torch.einsum("tgd,ld->gtl", q[:, h * group: (h + 1) * group], k[h]) / math.sqrt(case["dim"])
            w = w.masked_fill(hidden, -math.inf)
            total = torch.logsumexp(w, -1)
            rows.append(torch.einsum("gtl,ld->tgd", (w - total[..., None]).exp(), v[h]))
            logs.append(total.t())
        outs.append(torch.cat(rows, 1))
        sums.append(torch.cat(logs, 1))
    return torch.cat(outs), torch.cat(sums)


def _nearest(x, kind):
    """The nearest code's value, ties to even."""
    if kind == "int8":
        return torch.round(x).clamp(-127, 127)
    _, e = torch.frexp(x.abs())
    step = torch.exp2((e - 4).clamp(min=-9).double())  # 3 bits after the first; 2^-9 below the smallest normal
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(s):
    case = s["case"]
    ctx, new = _lengths(case)
    at, page, kind, half = _cu_host(new), case["page"], case["kv"], case["rot"] // 2
    ks, vs = s["ks"].double(), s["vs"].double()
    queries, keys, values = [], [], []

    def turn(x, lo):
        x, table = x.double(), s["rot"][lo: lo + x.shape[0]].double()
        z = torch.complex(table[..., 0], table[..., 1])[:, None]
        y = x.clone()
        i = torch.arange(half, device="cuda")
        one, two = (i, i + half) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
        turned = torch.complex(x[..., one], x[..., two]) * z
        y[..., one], y[..., two] = turned.real, turned.imag
        return y

    for b, (c, t) in enumerate(zip(ctx, new)):
        part = slice(int(at[b]), int(at[b + 1]))
        queries.append(turn(s["q"][part], c - t))
        first = (c - t) // page * page
        for codes, scales, x, got in ((s["k"], ks, turn(s["knew"][part], c - t), keys), (s["v"], vs, s["vnew"][part].double(), values)):
            had = c - t - first  # rows of the first page that are kept
            pieces = []
            n_pages = -(-(c - first) // page)
            padded = torch.zeros(n_pages * page, *x.shape[1:], dtype=torch.float64, device="cuda")
            padded[had: had + t] = x
            padded = padded.view(n_pages, page, case["hkv"], -1)
            ids = s["table"][b, first // page: first // page + n_pages].long()
            scale = padded.abs().amax((1, 3)) / TOP[kind]
            old = scales[ids[0]].clone()
            if had:
                scale[0] = torch.maximum(scale[0], old)
                was = codes.view(torch.int8)[ids[0]].view(codes.dtype).float().double()[:, :had]
                pieces.append((_nearest(was * (old / scale[0])[:, None, None], kind) * scale[0][:, None, None]).transpose(0, 1))
            wide = scale[:, None, :, None]
            stored = (_nearest(padded / wide.clamp(min=1e-300), kind) * wide).view(n_pages * page, case["hkv"], -1)
            pieces.append(stored[had: had + t])
            scales[ids] = scale
            got.append(torch.cat(pieces))
    return torch.cat(queries), torch.cat(keys), torch.cat(values), ks, vs
