"""Measured cases of the operators around a decoder layer's attention: the norms before and
after a block with its gate and residual scale, the append with rotary positions of several
axes, attention with a sliding window whose first tokens stay visible, and attention of a batch
that shares long prefixes.

``run`` computes an operator either by the library's entry points (``own = True``) or by its
plain form in elementary torch operations (``own = False``); ``exact`` computes the definition
in 64 bits.

Definitions
-----------
Norms: x = residual + scale * act(gate) * N_post(y), h = N(x). N of a row: rms
v / sqrt(mean(v^2) + eps) * weight, or layer (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) * weight
+ bias. Without a gate its factor is 1, without a post norm N_post(y) = y. h is taken from x before it is
rounded to its type.

Cache: codes [pages][kv heads][page][head dim], one 32-bit scale for each page and head; a value is
code * scale. Sequence b's token at position t lies in page block_table[b][t / page], row t % page.

Append: the new tokens of sequence b are its last ones, at places ctx_len[b] - new ... ctx_len[b] - 1
of the cache. A token has a rotary position on each axis (time, height, width); pair i of the rotated
elements is turned by row positions[axis of i][token] of a (cos, sin) table: (a, b) -> (a c - b s,
b c + a s), each product and sum rounded to 32 bits. Scales and codes, fl a rounding to 32 bits: a page's scale is the
larger of its old one (none, if its first row is new) and fl(largest new magnitude * fl(1 / top)),
top = 127 (int8) or 448 (e4m3); old codes of a page whose scale grew become round(fl(code * fl(old / new))),
new codes are round(fl(value / scale)), ties to even; a value is fl(code * scale).

Attention with a window w and s first tokens: the query of sequence b at position p sees the
positions t <= p with t > p - w or t < s.

Shared prefixes: sequences groups[j] .. groups[j + 1] - 1 all begin with the prefix_len[j] tokens in the
pages prefix_table[j]; their own tokens, ctx_len[b] of them, follow in the pages block_table[b]. The
query at a sequence's own position p sees the whole prefix and its own positions 0 .. p.

Outputs of attention are the softmax-weighted values and the natural log of the sum of exponentials.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BITS = {"f32": 4, "f16": 2, "bf16": 2}
TOP = {"int8": 127.0, "e4m3": 448.0}
EPS = 1e-6
SCALE = 0.75


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # One token of a decoding step between two blocks: the call's latency.
        {"name": "norm one token", "op": "norm", "tokens": 1, "width": 4096, "kind": "rms", "post": True, "gate": "none", "act": "none", "residual": "bf16", "x": "bf16"},
        # A decoding batch, rows that do not start on 16-byte boundaries, a gate for each channel.
        {"name": "norm batch ragged", "op": "norm", "tokens": 192, "width": 8177, "kind": "layer", "post": False, "gate": "channel", "act": "none", "residual": "f16", "x": "f16"},
        # Prompts: a 32-bit residual stream, a gate of each token's own: about 1.9 GB.
        {"name": "norm prompts", "op": "norm", "tokens": 16000, "width": 8192, "kind": "rms", "post": True, "gate": "token", "act": "silu", "residual": "f32", "x": "bf16"},
        # One text token for each of 4 sequences, behind images: the call's latency.
        {"name": "axes 4 tokens", "op": "append", "seqs": 4, "new": 1, "ctx": 700, "hq": 32, "hkv": 8, "dim": 128, "page": 16, "kv": "int8", "x": "bf16", "rot": 128, "pairs": "half", "order": "blocks"},
        # One token for each of 192 sequences, part of the head rotated, axes in turn over neighbouring pairs.
        {"name": "axes batch 192", "op": "append", "seqs": 192, "new": 1, "ctx": 4000, "hq": 32, "hkv": 8, "dim": 128, "page": 64, "kv": "e4m3", "x": "f16", "rot": 64, "pairs": "interleaved", "order": "turns"},
        # Images of up to 4096 patches for 4 sequences that have some tokens already.
        {"name": "axes prompts", "op": "append", "seqs": 4, "new": 4096, "ctx": 5001, "hq": 32, "hkv": 8, "dim": 128, "page": 32, "kv": "int8", "x": "f32", "rot": 128, "pairs": "half", "order": "blocks"},
        # One sequence, a short window: the call's latency.
        {"name": "sinks one short", "op": "sinks", "seqs": 1, "q": 1, "ctx": 5000, "window": 300, "sinks": 4, "hq": 16, "hkv": 4, "dim": 64, "page": 16, "kv": "int8", "x": "bf16"},
        # 64 sequences longer than the window: about 1.1 GB of cache seen.
        {"name": "sinks batch 64", "op": "sinks", "seqs": 64, "q": 1, "ctx": 17000, "window": 8192, "sinks": 4, "hq": 64, "hkv": 8, "dim": 128, "page": 64, "kv": "e4m3", "x": "bf16"},
        # Checking up to 5 drafted tokens of 24 sequences at once, 32-bit; the visible first tokens end inside a page.
        {"name": "sinks drafts f32", "op": "sinks", "seqs": 24, "q": 5, "ctx": 9000, "window": 4096, "sinks": 70, "hq": 30, "hkv": 6, "dim": 128, "page": 32, "kv": "int8", "x": "f32"},
        # Four short sequences behind a short common prompt: the call's latency.
        {"name": "shared short", "op": "shared", "groups": 1, "seqs": 4, "q": 1, "prefix": 1000, "ctx": 90, "hq": 16, "hkv": 4, "dim": 64, "page": 16, "kv": "e4m3", "x": "f16"},
        # 64 conversations behind one document of 32768 tokens.
        {"name": "shared batch 64", "op": "shared", "groups": 1, "seqs": 64, "q": 1, "prefix": 32768, "ctx": 700, "hq": 64, "hkv": 8, "dim": 128, "page": 64, "kv": "int8", "x": "bf16"},
        # Checking up to 5 drafted tokens of 40 sequences behind three prompts of different lengths, 32-bit.
        {"name": "shared drafts f32", "op": "shared", "groups": 3, "seqs": 40, "q": 5, "prefix": 8001, "ctx": 600, "hq": 30, "hkv": 6, "dim": 128, "page": 32, "kv": "int8", "x": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "append", "sinks", "shared"))
    x = rng.choice(("f32", "f16", "bf16"))
    if op == "norm":
        width = _log(rng, 64, 16384)
        gate = rng.choice(("none", "channel", "token"))
        return {"op": op, "tokens": _log(rng, 1, min(16000, 16000 * 4096 // width)), "width": width, "kind": rng.choice(("rms", "layer")), "post": rng.random() < 0.5,
                "gate": gate, "act": "none" if gate == "none" else rng.choice(("none", "sigmoid", "silu")), "residual": rng.choice((x, x, "f32")), "x": x}
    kv = rng.choice(("int8", "e4m3"))
    dim, page = rng.choice((64, 128, 128, 256)), rng.choice((16, 32, 64, 128))
    hkv = rng.choice((1, 2, 4, 5, 8))
    if op == "append":
        seqs = _log(rng, 1, 192)
        new = 1 if rng.random() < 0.5 else max(1, _log(rng, 1, 4096) // seqs)
        hq = hkv * rng.choice((2, 5, 8))
        return {"op": op, "seqs": seqs, "new": new, "ctx": new + _log(rng, 1, 4000), "hq": hq, "hkv": hkv, "dim": dim, "page": page, "kv": kv, "x": x,
                "rot": rng.choice((dim, dim, dim // 2)), "pairs": rng.choice(("half", "interleaved")), "order": rng.choice(("blocks", "turns"))}
    group = rng.choice((1, 2, 4, 5, 8))
    q = rng.choice((1, 1, 1, 2, 4, 8))
    seqs = _log(rng, 1, 64)
    if op == "sinks":
        window = _log(rng, 16, 16384)
        # what a sequence sees, as in the largest listed case
        window = max(16, min(window, 64 * 8192 * 1024 // (seqs * hkv * dim * max(1, q * group // 8))))
        ctx = min(max(8, _log(rng, window // 2 + 8, 4 * window + 100)), 64 * 17000 * 1024 // (seqs * hkv * dim))
        return {"op": op, "seqs": seqs, "q": q, "ctx": ctx, "window": window, "sinks": _log(rng, 1, 200), "hq": hkv * group, "hkv": hkv, "dim": dim, "page": page, "kv": kv, "x": x}
    # scores no more than in the largest listed case; a prefix of 32-bit queries counts twice
    most = 64 * 64 * 32768 * 128 // (hkv * group * seqs * q * dim * (2 if x == "f32" else 1))
    return {"op": op, "groups": rng.randint(1, min(4, seqs)), "seqs": seqs, "q": q, "prefix": max(16, min(_log(rng, 100, 65536), most)),
            "ctx": max(8, min(_log(rng, 10, 4000), most)), "hq": hkv * group, "hkv": hkv, "dim": dim, "page": page, "kv": kv, "x": x}


# ------------------------------------------------------ lengths, by the case
def _share(b):
    """0.5 .. 1, spread evenly over the sequences, the first one 1."""
    return 1.0 - 0.5 * ((b * 0.6180339887498949) % 1.0)


def _lengths(case):
    """(ctx, new) of each sequence; new: the tokens appended or queried."""
    ctx = [max(1, int(case["ctx"] * _share(b))) for b in range(case["seqs"])]
    new = [max(1, int(case["new" if case["op"] == "append" else "q"] * _share(3 * b))) for b in range(case["seqs"])]
    return [max(c, t) for c, t in zip(ctx, new)], new


def _groups(case):
    """Offsets of the groups' sequences (uneven shares, one at least) and their prefixes' lengths."""
    n, seqs = case["groups"], case["seqs"]
    weights = [_share(5 * j + 1) for j in range(n)]
    total, at, run_ = sum(weights), [0], 0.0
    for j, w in enumerate(weights):
        run_ += w
        at.append(seqs if j == n - 1 else min(max(at[-1] + 1, int(seqs * run_ / total)), seqs - (n - 1 - j)))
    return at, [max(1, int(case["prefix"] * _share(j))) for j in range(n)]


def _append_reads(case):
    """First position and count, for each sequence, of the tokens in the pages that an append touches."""
    ctx, new = _lengths(case)
    first = [(c - t) // case["page"] * case["page"] for c, t in zip(ctx, new)]
    return first, [c - f for c, f in zip(ctx, first)]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(counts):
    return _i32([0] + list(np.cumsum(counts)))


# --------------------------------------------------------------- the inputs
def _rotation_table(rows, rot):
    """cos and sin of position * 10000^(-2 i / rot), from 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.stack((angle.cos(), angle.sin()), -1).float().contiguous()


def _axis_of_pairs(case):
    """The axis (0 time, 1 height, 2 width) of each rotated pair: a quarter, three eighths and three eighths of them
    one after the other, or in turns."""
    half = case["rot"] // 2
    if case["order"] == "turns":
        return [i % 3 for i in range(half)]
    t = half // 4
    h = (half - t) // 2
    return [0] * t + [1] * h + [2] * (half - t - h)


GRID = (23, 31)  # rows and columns of an image's patches


def _positions(case):
    """Three rotary positions of each new token: one token continues as text (the same on all axes), more are
    images one after the other, in patches."""
    ctx, new = _lengths(case)
    out = []
    for c, t in zip(ctx, new):
        i = np.arange(t)
        if t == 1:
            out.append(np.full((3, 1), c // 2))
        else:
            out.append((c - t) // 2 + np.stack((i // (GRID[0] * GRID[1]), i // GRID[1] % GRID[0], i % GRID[1])))
    return np.concatenate(out, 1).astype(np.int32)


def _tables(lengths, page, order, start):
    """A table of each sequence's pages, from place `start` of the order on; unused places hold page 0."""
    used = [-(-n // page) for n in lengths]
    width = max(used)
    table = torch.zeros(len(lengths), width, dtype=torch.int32, device="cuda")
    live = torch.arange(width, device="cuda")[None, :] < _i32(used)[:, None]
    table[live] = order[start: start + sum(used)]
    return table, start + sum(used)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = {"generator": g, "device": "cuda"}
    s = {"case": case}
    x = DTYPES[case["x"]]
    if case["op"] == "norm":
        tokens, width = case["tokens"], case["width"]
        s["y"] = torch.randn(tokens, width, dtype=x, **kw)
        s["r"] = torch.randn(tokens, width, dtype=DTYPES[case["residual"]], **kw).mul_(3)
        s["gate"] = {"none": lambda: None, "channel": lambda: torch.randn(width, dtype=x, **kw), "token": lambda: torch.randn(tokens, width, dtype=x, **kw)}[case["gate"]]()
        for name, there in (("w", True), ("b", case["kind"] == "layer"), ("pw", case["post"]), ("pb", case["post"] and case["kind"] == "layer")):
            s[name] = (torch.randn(width, **kw) * 0.2 + (name[-1] == "w")).to(x) if there else None
        return s
    seqs, hkv, dim, page = case["seqs"], case["hkv"], case["dim"], case["page"]
    ctx, new = _lengths(case)
    lengths, prefixes = list(ctx), []
    if case["op"] == "shared":
        at, prefixes = _groups(case)
        s["groups"], s["plen"] = _i32(at), _i32(prefixes)
    pages = sum(-(-c // page) for c in lengths + prefixes) + 3
    # every sequence and prefix its own pages, in random order
    order = torch.randperm(pages, **kw).to(torch.int32)
    s["table"], used = _tables(ctx, page, order, 0)
    if prefixes:
        s["ptable"], _ = _tables(prefixes, page, order, used)
    codes = []
    for _ in range(2):  # keys, values
        if case["kv"] == "int8":
            c = torch.randn(pages, hkv, page, dim, dtype=torch.float16, **kw).mul_(38).clamp_(-127, 127).round_().to(torch.int8)
        else:
            c = torch.randn(pages, hkv, page, dim, dtype=torch.float16, **kw).mul_(110).clamp_(-448, 448).to(torch.float8_e4m3fn)
        codes.append(c)
    s["k"], s["v"] = codes
    s["ks"], s["vs"] = (((0.7 + 0.6 * torch.rand(pages, hkv, **kw)) * (3.3 / TOP[case["kv"]])).contiguous() for _ in range(2))
    s["ctx"], s["cu"], s["total"], s["most"] = _i32(ctx), _cu(new), sum(new), max(new)
    append = case["op"] == "append"
    # queries (keys and values) are parts of one product's output rows
    rows = torch.randn(sum(new), case["hq"] + (2 * hkv if append else 0), dim, **kw)
    if not append:
        rows *= 1.5
    rows = rows.to(x)
    s["q"] = rows[:, : case["hq"]]
    if append:
        s["knew"], s["vnew"] = rows[:, case["hq"]: case["hq"] + hkv], rows[:, case["hq"] + hkv:]
        s["rot"] = _rotation_table(max(ctx) + max(GRID) + 1, case["rot"])
        s["pos"] = torch.from_numpy(_positions(case)).cuda()
        s["axis"] = _i32(_axis_of_pairs(case))
        first, count = _append_reads(case)
        s["first"], s["rcu"], s["rmost"], s["rtotal"] = _i32(first), _cu(count), max(count), sum(count)
    if own:
        import implicit_gemm_convolution_gb300 as om
        s["cache"] = om.PagedKVCache(s["k"], s["v"], s["ks"], s["vs"])
        if not append:
            s["lse"] = torch.empty(s["total"], case["hq"], dtype=torch.float32, device="cuda")
        if case["op"] == "sinks":
            s["ws"] = om.new_kv_workspace(s["cache"], case["hq"], s["most"])
        if case["op"] == "shared":
            s["ws"] = om.new_shared_workspace(s["cache"], case["hq"], s["most"], s["total"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import implicit_gemm_convolution_gb300 as om
    case = s["case"]
    if case["op"] == "norm":
        return om.block_norm(s["y"], s["r"], s["w"], s["b"], post_weight=s["pw"], post_bias=s["pb"], gate=s["gate"], activation=case["act"], scale=SCALE, norm=case["kind"], eps=EPS)
    if case["op"] == "append":
        q = om.kv_append(s["cache"], s["q"], s["knew"], s["vnew"], s["rot"], s["table"], s["ctx"], s["cu"], s["most"], pairs=case["pairs"],
                         positions=s["pos"], pair_axis=s["axis"])
        # the cache as the values it stands for
        k, v = om.kv_read(s["cache"], s["table"], s["first"], s["rcu"], s["rmost"], s["rtotal"])
        return q, k, v, s["ks"], s["vs"]
    if case["op"] == "sinks":
        out = om.kv_attention(s["cache"], s["q"], s["table"], s["ctx"], s["cu"], s["most"], window=case["window"], sinks=case["sinks"], lse=s["lse"], workspace=s["ws"])
    else:
        out = om.kv_shared_attention(s["cache"], s["q"], s["ptable"], s["plen"], s["groups"], s["table"], s["ctx"], s["cu"], s["most"], lse=s["lse"], workspace=s["ws"])
    return out, s["lse"]


def _run_plain(s):
    return {"norm": _plain_norm, "append": _plain_append, "sinks": _plain_sinks, "shared": _plain_shared}[s["case"]["op"]](s)


def _normed(v, kind, w, b):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    if w is not None:
        v = v * w.float()
    return v + b.float() if b is not None else v


def _plain_norm(s):
    case = s["case"]
    v = s["y"].float()
    if case["post"]:
        v = _normed(v, case["kind"], s["pw"], s["pb"])
    if case["gate"] != "none":
        g = s["gate"].float()
        if case["act"] != "none":
            t = 1.0 / (1.0 + (-g).exp())
            g = g * t if case["act"] == "silu" else t
        v = v * g
    v = s["r"].float() + SCALE * v
    return v.to(s["r"].dtype), _normed(v, case["kind"], s["w"], s["b"]).to(s["y"].dtype)


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


def _round_codes(x, kind):
    x = x.clamp(-TOP[kind], TOP[kind])
    return x.round().to(torch.int8) if kind == "int8" else x.to(torch.float8_e4m3fn)


def _to_codes(x, scale, kind):
    return _round_codes(torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0), kind)


def _plain_append(s):
    case = s["case"]
    page, kind, hkv = case["page"], case["kv"], case["hkv"]
    counts = s["cu"][1:] - s["cu"][:-1]
    b, place = _tokens(s, s["ctx"] - counts, s["cu"], s["total"])
    # a token's row of the table, put together from its axes' rows
    cs = s["rot"][s["pos"].long()[s["axis"].long()].t(), torch.arange(case["rot"] // 2, device="cuda")]
    q = _rotate(s["q"], cs, case["rot"], case["pairs"]).to(s["q"].dtype)
    at, row = s["table"].long()[b, place // page], place % page
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
    b, place = _tokens(s, s["first"], s["rcu"], s["rtotal"])
    at, row = s["table"].long()[b, place // page], place % page

    def part(codes, scales):
        c = codes.view(torch.int8)[at[:, None], heads, row[:, None]].view(codes.dtype)
        return c.float() * scales[at][:, :, None]

    return q, part(s["k"], s["ks"]), part(s["v"], s["vs"]), s["ks"], s["vs"]


def _whole(s, table, codes, scales):
    """Keys or values of the tables' pages: tables x heads x positions x dim."""
    t = table.long()
    c = codes.view(torch.int8)[t].view(codes.dtype).float().mul_(scales[t][..., None, None])
    return c.transpose(1, 2).reshape(t.shape[0], s["case"]["hkv"], -1, s["case"]["dim"])


def _softmax(scores, values):
    """Largest score, sum of exponentials and weighted values of scores (..., rows, positions)."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    e = scores.sub_(top).exp_()
    return top, e.sum(-1, keepdim=True), e @ values


def _padded(s):
    """Queries by sequence, seqs x heads x (heads of a group, queries) x dim, their own positions (-1: none),
    and the places of the tokens in them."""
    case = s["case"]
    seqs, hq, hkv, dim, most = case["seqs"], case["hq"], case["hkv"], case["dim"], s["most"]
    counts = s["cu"][1:] - s["cu"][:-1]
    b, pos = _tokens(s, s["ctx"] - counts, s["cu"], s["total"])
    i = torch.arange(s["total"], device="cuda") - s["cu"].long()[b]
    q = torch.zeros(seqs, most, hq, dim, device="cuda").index_put_((b, i), s["q"].float())
    p = torch.full((seqs, most), -1, device="cuda").index_put_((b, i), pos)
    return q.transpose(1, 2).reshape(seqs, hkv, (hq // hkv) * most, dim), p, b, i


def _plain_own(s, window, sinks):
    """Largest score, sum and weighted values of each token and head over its sequence's own tokens."""
    case = s["case"]
    seqs, hq, most = case["seqs"], case["hq"], s["most"]
    q, p, b, i = _padded(s)
    scores = (q @ _whole(s, s["table"], s["k"], s["ks"]).transpose(2, 3)).mul_(case["dim"] ** -0.5)
    t = torch.arange(scores.shape[-1], device="cuda")
    seen = t <= p[..., None]
    if window:
        seen &= (t > p[..., None] - window) | (t < sinks)
    scores.view(seqs, hq, most, -1).masked_fill_(~seen[:, None], -math.inf)
    got = _softmax(scores, _whole(s, s["table"], s["v"], s["vs"]))
    return [x.reshape(seqs, hq, most, -1).transpose(1, 2)[b, i] for x in got]


def _plain_sinks(s):
    top, total, out = _plain_own(s, s["case"]["window"], s["case"]["sinks"])
    return (out / total).to(s["q"].dtype), (total.log() + top)[..., 0]


def _plain_shared(s):
    case = s["case"]
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    top, total, out = _plain_own(s, 0, 0)
    at, prefixes = _groups(case)
    cu = np.concatenate([[0], np.cumsum(_lengths(case)[1])])
    for j, n in enumerate(prefixes):
        part = slice(int(cu[at[j]]), int(cu[at[j + 1]]))
        q = s["q"][part].float().view(-1, hkv, hq // hkv, dim).transpose(0, 1).reshape(hkv, -1, dim)
        table = s["ptable"][j: j + 1]
        keys, values = (_whole(s, table, c, k)[0, :, :n] for c, k in ((s["k"], s["ks"]), (s["v"], s["vs"])))
        got = _softmax((q @ keys.transpose(1, 2)).mul_(dim ** -0.5), values)
        ptop, ptotal, pout = (x.view(hkv, -1, hq // hkv, x.shape[-1]).transpose(0, 1).reshape(-1, hq, x.shape[-1]) for x in got)
        best = torch.maximum(top[part], ptop)
        a, b = (top[part] - best).exp(), (ptop - best).exp()
        out[part] = out[part] * a + pout * b
        total[part] = total[part] * a + ptotal * b
        top[part] = best
    return (out / total).to(s["q"].dtype), (total.log() + top)[..., 0]


# ---------------------------------------------------------- the bare work
def work(case):
    x = BITS[case["x"]]
    if case["op"] == "norm":
        one = case["tokens"] * case["width"]
        vectors = 1 + (case["kind"] == "layer") + case["post"] * (1 + (case["kind"] == "layer")) + (case["gate"] == "channel")
        return {"bytes": one * (2 * x + 2 * BITS[case["residual"]] + (x if case["gate"] == "token" else 0)) + vectors * case["width"] * x,
                "flops": one * (6 + 5 * case["post"] + 2 * (case["gate"] != "none"))}
    ctx, new = _lengths(case)
    hq, hkv, dim, page = case["hq"], case["hkv"], case["dim"], case["page"]
    if case["op"] == "append":
        first, count = _append_reads(case)
        old = sum(count) - sum(new)
        one = sum(new) * dim
        rewritten = 2 * hkv * dim * 2 * old  # the codes of a page whose scale grows, once in and once out
        values = sum(count) * hkv * dim * 2 * (1 + 4)
        return {"bytes": one * (2 * hq + 2 * hkv) * x + one * hkv * 2 + sum(new) * (case["rot"] * 4 + 12) + rewritten + values,
                "flops": one * (hq + hkv) * 3 + one * hkv * 4}
    rows = sum(new) * hq * (2 * dim * x + 4)
    if case["op"] == "sinks":
        w, f = case["window"], case["sinks"]
        pairs = sum(min(p, w) + min(f, max(0, p - w)) for c, t in zip(ctx, new) for p in range(c - t + 1, c + 1))
        seen = [min(c, w + t - 1) + min(f, max(0, c - w - t + 1)) for c, t in zip(ctx, new)]
        spots = sum(-(-r // page) for r in seen)
        return {"bytes": sum(seen) * hkv * dim * 2 + spots * (hkv * 8 + 4) + rows, "flops": 4 * pairs * hq * dim}
    at, prefixes = _groups(case)
    pairs = sum(c - t + i + 1 for c, t in zip(ctx, new) for i in range(t))
    pairs += sum(n * sum(new[at[j]: at[j + 1]]) for j, n in enumerate(prefixes))
    spots = sum(-(-n // page) for n in ctx + prefixes)
    return {"bytes": (sum(ctx) + sum(prefixes)) * hkv * dim * 2 + spots * (hkv * 8 + 4) + rows, "flops": 4 * pairs * hq * dim}


# --------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    global own
    kept, own = own, False
    s = prepare(case, seed)
    own = kept
    return {"norm": _exact_norm, "append": _exact_append, "sinks": _exact_sinks, "shared": _exact_shared}[case["op"]](s)


def _exact_norm(s):
    case = s["case"]
    xs, hs = [], []

    def over(v, w, b):
        if case["kind"] == "layer":
            var, mean = torch.var_mean(v, -1, correction=0, keepdim=True)
        else:
            var, mean = v.square().mean(-1, keepdim=True), 0.0
        v = (v - mean) / torch.sqrt(var + EPS) * w.double()
        return v if b is None else v + b.double()

    step = max(1, (1 << 25) // case["width"])
    for i in range(0, case["tokens"], step):
        v = s["y"][i: i + step].double()
        if case["post"]:
            v = over(v, s["pw"], s["pb"])
        if case["gate"] != "none":
            g = (s["gate"] if case["gate"] == "channel" else s["gate"][i: i + step]).double()
            v = v * {"none": lambda: g, "sigmoid": lambda: torch.sigmoid(g), "silu": lambda: g * torch.sigmoid(g)}[case["act"]]()
        v = s["r"][i: i + step].double() + SCALE * v
        xs.append(v)
        hs.append(over(v, s["w"], s["b"]))
    return torch.cat(xs), torch.cat(hs)


def _sequence(s, ids, n):
    """Keys and values of the first n positions of a table's pages: heads x positions x dim."""
    ids = ids[: -(-n // s["case"]["page"])].long()
    out = []
    for codes, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        c = codes.view(torch.int8)[ids].view(codes.dtype).to(torch.float32).double() * scales[ids].double()[:, :, None, None]
        out.append(c.transpose(0, 1).flatten(1, 2)[:, :n])
    return out


def _exact_rows(s, b, lo, hi, k, v, hidden):
    """Outputs and log sums of the tokens lo .. hi - 1 over keys and values k, v; hidden: queries x positions."""
    case = s["case"]
    group = case["hq"] // case["hkv"]
    q = s["q"][lo:hi].double()
    rows, logs = [], []
    for h in range(case["hkv"]):
        w = torch.einsum("tgd,ld->gtl", q[:, h * group: (h + 1) * group], k[h]) / math.sqrt(case["dim"])
        w = w.masked_fill(hidden, -math.inf)
        total = torch.logsumexp(w, -1)
        rows.append(torch.einsum("gtl,ld->tgd", (w - total[..., None]).exp(), v[h]))
        logs.append(total.t())
    return torch.cat(rows, 1), torch.cat(logs, 1)


def _exact_sinks(s):
    case = s["case"]
    ctx, new = _lengths(case)
    at = np.concatenate([[0], np.cumsum(new)])
    got = []
    for b, (c, t) in enumerate(zip(ctx, new)):
        here, there = torch.arange(c - t, c, device="cuda")[:, None], torch.arange(c, device="cuda")[None, :]
        seen = (there <= here) & ((there > here - case["window"]) | (there < case["sinks"]))
        got.append(_exact_rows(s, b, int(at[b]), int(at[b + 1]), *_sequence(s, s["table"][b], c), ~seen))
    return tuple(torch.cat([g[j] for g in got]) for j in range(2))


def _exact_shared(s):
    case = s["case"]
    ctx, new = _lengths(case)
    offsets = np.concatenate([[0], np.cumsum(new)])
    at, prefixes = _groups(case)
    got = []
    for j, n in enumerate(prefixes):
        pk, pv = _sequence(s, s["ptable"][j], n)
        for b in range(at[j], at[j + 1]):
            c, t = ctx[b], new[b]
            k, v = _sequence(s, s["table"][b], c)
            hidden = torch.arange(n + c, device="cuda")[None, :] > torch.arange(n + c - t, n + c, device="cuda")[:, None]
            got.append(_exact_rows(s, b, int(offsets[b]), int(offsets[b + 1]), torch.cat((pk, k), 1), torch.cat((pv, v), 1), hidden))
    return tuple(torch.cat([g[i] for g in got]) for i in range(2))


def _nearest(x, kind):
    """The nearest code's value, ties to even."""
    if kind == "int8":
        return torch.round(x).clamp(-127, 127)
    _, e = torch.frexp(x.abs())
    step = torch.exp2((e - 4).clamp(min=-9).double())  # 3 bits after the first; 2^-9 below the smallest normal
    return (torch.round(x / step) * step).clamp(-448, 448)


def _fl(x):
    """Rounded to 32 bits: products, sums and quotients of such numbers in 64 bits round there as if taken exactly."""
    return x.float().double()


def _exact_append(s):
    case = s["case"]
    ctx, new = _lengths(case)
    offsets, page, kind, half = np.concatenate([[0], np.cumsum(new)]), case["page"], case["kv"], case["rot"] // 2
    ks, vs = s["ks"].double(), s["vs"].double()
    queries, keys, values = [], [], []
    axis = _axis_of_pairs(case)

    def turn(x):
        x = x.double()
        cs = torch.stack([s["rot"].double()[s["pos"][axis[i]].long(), i] for i in range(half)], 1)[:, None]
        y = x.clone()
        i = torch.arange(half, device="cuda")
        one, two = (i, i + half) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
        c, d = cs[..., 0], cs[..., 1]
        y[..., one] = _fl(_fl(x[..., one] * c) - _fl(x[..., two] * d))
        y[..., two] = _fl(_fl(x[..., two] * c) + _fl(x[..., one] * d))
        return y

    turned_q, turned_k = turn(s["q"]), turn(s["knew"])
    step = _fl(torch.tensor(1.0 / TOP[kind], dtype=torch.float64)).item()
    for b, (c, t) in enumerate(zip(ctx, new)):
        part = slice(int(offsets[b]), int(offsets[b + 1]))
        queries.append(turned_q[part])
        first = (c - t) // page * page
        for codes, scales, x, got in ((s["k"], ks, turned_k[part], keys), (s["v"], vs, s["vnew"][part].double(), values)):
            had = c - t - first  # rows of the first page that are kept
            pieces = []
            n_pages = -(-(c - first) // page)
            padded = torch.zeros(n_pages * page, *x.shape[1:], dtype=torch.float64, device="cuda")
            padded[had: had + t] = x
            padded = padded.view(n_pages, page, case["hkv"], -1)
            ids = s["table"][b, first // page: first // page + n_pages].long()
            scale = _fl(padded.abs().amax((1, 3)) * step)
            old = scales[ids[0]].clone()
            if had:
                scale[0] = torch.maximum(scale[0], old)
                was = codes.view(torch.int8)[ids[0]].view(codes.dtype).float().double()[:, :had]
                pieces.append(_fl(_nearest(_fl(was * _fl(old / scale[0])[:, None, None]), kind) * scale[0][:, None, None]).transpose(0, 1))
            wide = scale[:, None, :, None]
            stored = _fl(_nearest(_fl(padded / wide.clamp(min=1e-300)), kind) * wide).view(n_pages * page, case["hkv"], -1)
            pieces.append(stored[had: had + t])
            scales[ids] = scale
            got.append(torch.cat(pieces))
    return torch.cat(queries), torch.cat(keys), torch.cat(values), ks, vs
