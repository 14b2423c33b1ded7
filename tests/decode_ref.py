"""Plain 64-bit (and, where outputs have one bit pattern, 32-bit) references of
the decoding operators, in numpy."""
import numpy as np
import torch

TOP = {"int8": 127.0, "e4m3": 448.0}
CODE_DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a unit in the last place, relative
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}


def f64(t):
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64) if t.dtype != torch.float64 else t.cpu().numpy()


def e4m3_values():
    return torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)


def code_values(codes):
    """The values of a tensor of codes (numpy float64)."""
    raw = codes.detach().view(torch.int8).cpu().numpy()
    return raw.astype(np.float64) if codes.dtype == torch.int8 else e4m3_values()[raw.view(np.uint8)]


def w4_weights(u, s, z, k, group):
    u, s = u.cpu().numpy(), f64(s)
    codes = np.stack((u & 15, u >> 4), -1).reshape(u.shape[0], -1)[:, :k].astype(np.float64)
    at = np.arange(k) // group
    zero = z.cpu().numpy().astype(np.float64)[:, at] if z is not None else 8.0
    return (codes - zero) * s[:, at]


def attention(q, k_codes, v_codes, ks, vs, table, ctx, cu, scale, window, page):
    """out, lse, and for each output sum p |v| and the largest sum |q||k| of its
    scores; arrays [tokens][q heads][dim], [tokens][q heads], ..."""
    T, hq, dim = q.shape
    hkv = k_codes.shape[1]
    g = hq // hkv
    out, lse = np.zeros((T, hq, dim)), np.full((T, hq), -np.inf)
    mag, sc = np.zeros((T, hq, dim)), np.zeros((T, hq))
    for b in range(len(ctx)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            p = ctx[b] - n + i
            lo = max(0, p - window + 1) if window else 0
            pos = [t for t in range(lo, p + 1) if t // page < table.shape[1] and 0 <= table[b][t // page] < k_codes.shape[0]]
            if not pos:
                continue
            pos = np.array(pos)
            ids, rows = table[b][pos // page], pos % page
            for h in range(hq):
                kk = k_codes[ids, h // g, rows] * ks[ids, h // g][:, None]
                vv = v_codes[ids, h // g, rows] * vs[ids, h // g][:, None]
                qq = q[cu[b] + i, h]
                s = scale * (kk @ qq)
                m = s.max()
                e = np.exp(s - m)
                w = e / e.sum()
                t = cu[b] + i
                out[t, h] = w @ vv
                lse[t, h] = m + np.log(e.sum())
                mag[t, h] = w @ np.abs(vv)
                sc[t, h] = scale * (np.abs(kk) @ np.abs(qq)).max()
    return out, lse, mag, sc


def rotate(x, table, pos, rot, interleaved):
    """x [tokens][heads][dim] float32, every product and sum rounded to float32."""
    y = x.astype(np.float32).copy()
    for t, p in enumerate(pos):
        if rot == 0:
            continue
        cs = table[p] if 0 <= p < table.shape[0] else np.full((rot // 2, 2), np.nan, np.float32)
        c, s = cs[:, 0].astype(np.float32), cs[:, 1].astype(np.float32)
        i = np.arange(rot // 2)
        one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = x[t][:, one].astype(np.float32), x[t][:, two].astype(np.float32)
        with np.errstate(invalid="ignore", over="ignore"):
            y[t][:, one] = a * c - b * s
            y[t][:, two] = b * c + a * s
    return y


def encode(x, kind):
    """The nearest codes (as int8 bytes) of float32 values."""
    x = np.clip(x.astype(np.float32), -np.float32(TOP[kind]), np.float32(TOP[kind]))
    if kind == "int8":
        return np.rint(x).astype(np.int8)
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.float8_e4m3fn).view(torch.int8).numpy()


def append(codes, scales, new, table, ctx, cu, page, kind):
    """The cache after the append of `new` [tokens][heads][dim] (float32, rotated):
    (raw int8 codes, scales), copies; codes as a raw int8 array, in float32 arithmetic."""
    codes, scales = codes.copy(), scales.copy()
    values = e4m3_values().astype(np.float32)
    one = np.float32(1.0) / np.float32(TOP[kind])
    for b in range(len(ctx)):
        n = cu[b + 1] - cu[b]
        start = ctx[b] - n
        for j in range(max(start, 0) // page, -(-ctx[b] // page) if ctx[b] > 0 and n else 0):
            if j >= table.shape[1] or not 0 <= table[b][j] < codes.shape[0]:
                continue
            pid = table[b][j]
            lo, hi = max(start, j * page, 0), min(ctx[b], (j + 1) * page)
            had = lo - j * page
            for h in range(codes.shape[1]):
                x = new[cu[b] + lo - start: cu[b] + hi - start, h]
                old = np.float32(scales[pid, h]) if had else np.float32(0)
                with np.errstate(invalid="ignore", over="ignore"):
                    top = np.abs(x).max()
                    bad = not np.isfinite(top) or not np.isfinite(old)
                    grown = np.float32(np.nan) if bad else max(old, np.float32(top * one))
                if had and (bad or grown != old):
                    raw = codes[pid, h, :had]
                    was = raw.astype(np.float32) if kind == "int8" else values[raw.view(np.uint8)]
                    codes[pid, h, :had] = encode(was * np.float32(0 if bad else old / grown), kind) if not bad else 0
                scales[pid, h] = grown
                codes[pid, h, had: had + hi - lo] = 0 if bad or grown == 0 else encode(x / grown, kind)
    return codes, scales
