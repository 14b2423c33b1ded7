"""The fused norms on the GPU against the formula in 64 bits.

Tolerances, u = 2^-24: a sum of n terms of one sign is taken in chains of at most 32 terms and 10 steps of a tree, so
it is off by 43 u of itself at most (64 u leaves room for its division and root); differences from a mean carry the
mean's error, 64 u of the mean magnitude, as they are; every product, sum and quotient after that adds u; the
exponential is within 2 units (4 u), so a gate's factor within 8 u. What x is off by moves h as the norm's
derivative does. Each output adds half a unit of its type.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests import decode_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


def normed(v, tol, kind, w, b, eps):
    """N(v) and its tolerance, of v known to `tol`."""
    mean, mean_tol = 0.0, 0.0
    if kind == "layer":
        mean = v.mean(-1, keepdims=True)
        mean_tol = 64 * U * np.abs(v).mean(-1, keepdims=True) + tol.mean(-1, keepdims=True)
    d, d_tol = v - mean, tol + mean_tol
    d_tol = d_tol + U * (np.abs(d) if kind == "layer" else 0.0)
    q = (d * d).mean(-1, keepdims=True) + eps
    inv = 1.0 / np.sqrt(q)
    # d(1 / sqrt(q)) = inv / (2 q) dq
    inv_tol = inv * (64 * U + ((np.abs(d) + 0.5 * d_tol) * d_tol).mean(-1, keepdims=True) / q)
    w = 1.0 if w is None else w
    h = d * inv * w
    h_tol = np.abs(w) * (d_tol * inv + np.abs(d) * inv_tol + d_tol * inv_tol) + 3 * U * np.abs(h)
    if b is not None:
        h = h + b
        h_tol = h_tol + U * np.abs(h)
    return h, h_tol


def check(got, y, r=None, w=None, b=None, pw=None, pb=None, gate=None, act=None, scale=1.0, kind="rms", post=None, eps=1e-6, x="f32", rx=None, normed_too=True):
    f = lambda t: None if t is None else ref.f64(t)
    scale, eps = float(np.float32(scale)), float(np.float32(eps))
    with np.errstate(over="ignore", invalid="ignore"):
        v = f(y)
        tol = np.zeros_like(v)
        if post or (post is None and (pw is not None or pb is not None)):
            v, tol = normed(v, tol, kind, f(pw), f(pb), eps)
        if gate is not None:
            g = f(gate)
            t = 1.0 / (1.0 + np.exp(-g))
            a = {None: lambda: g, "none": lambda: g, "sigmoid": lambda: t, "silu": lambda: np.where(np.isneginf(g), 0.0, g * t)}[act]()
            # factors that leave the range of 32 bits are 0
            tol = tol * np.abs(a) + np.abs(v) * (9 * U * np.abs(a) + 2.0 ** -120)
            v = v * a
        tol = abs(scale) * tol + U * np.abs(scale * v)
        v = scale * v
        if r is not None:
            v = f(r) + v
        tol = tol + U * np.abs(v) + 2.0 ** -149
        if got[0] is not None:
            off = np.abs(f(got[0]) - v)
            t = tol + 1.001 * ref.UNIT[rx or x] * (np.abs(v) + tol) + ref.TINY[rx or x]
            assert (off <= t).all(), f"x: {float((off / t).max())} of the tolerance"
        if normed_too:
            h, tol = normed(v, tol, kind, f(w), f(b), eps)
            off = np.abs(f(got[1]) - h)
            t = tol + 1.001 * ref.UNIT[x] * (np.abs(h) + tol) + ref.TINY[x]
            assert (off <= t).all(), f"h: {float((off / t).max())} of the tolerance"


def inputs(tokens, width, x, rx, seed, gate=None, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    T = ref.TORCH[x]
    d = {"y": (rn(tokens, width) * spread + 0.5).to(T), "r": (3 * rn(tokens, width)).to(ref.TORCH[rx or x])}
    d["gate"] = {None: lambda: None, "channel": lambda: rn(width).to(T), "token": lambda: (4 * rn(tokens, width)).to(T)}[gate]()
    for name in ("w", "b", "pw", "pb"):
        d[name] = (0.3 * rn(width) + (name[-1] == "w")).to(T)
    return d


SHAPES = [(1, 1), (1, 8), (3, 7), (2, 33), (5, 64), (4, 1000), (700, 300), (9, 1024), (1, 4096), (310, 4096), (3, 8177), (2, 8192), (320, 8200),
          (1, 16384), (2, 16383), (3, 32768), (2, 32767), (310, 20000), (2000, 96)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("x,rx", [("f32", None), ("f16", None), ("bf16", None), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("tokens,width", SHAPES)
def test_after_and_before_a_block(tokens, width, x, rx, kind):
    i = SHAPES.index((tokens, width))
    gate, act = [(None, None), ("channel", None), ("token", "silu"), ("token", "sigmoid"), ("channel", "silu")][(i + (kind == "rms")) % 5]
    d = inputs(tokens, width, x, rx, 31 * i + 7, gate)
    biased = kind == "layer"
    kw = dict(gate=d["gate"], scale=0.35)
    got = om.block_norm(d["y"], d["r"], d["w"], d["b"] if biased else None, post_weight=d["pw"] if i % 3 else None, post_bias=d["pb"] if biased and i % 2 else None,
                        post=None if i % 3 else bool(i % 2), activation=act, norm=kind, **kw)
    check(got, d["y"], d["r"], d["w"], d["b"] if biased else None, d["pw"] if i % 3 else None, d["pb"] if biased and i % 2 else None, act=act, kind=kind,
          post=None if i % 3 else bool(i % 2) or (biased and bool(i % 2)), x=x, rx=rx, **kw)


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_one_norm_alone(x):
    """Before a first block, without weights, and after a last one."""
    d = inputs(6, 520, x, None, 3)
    none, h = om.block_norm(d["y"], weight=d["w"])
    assert none is None
    check((None, h), d["y"], w=d["w"], x=x)
    check((None, om.block_norm(d["y"])[1]), d["y"], x=x)
    s, none = om.block_norm(d["y"], d["r"], post_weight=d["pw"], scale=-2.0, normed=False)
    assert none is None
    check((s, None), d["y"], d["r"], pw=d["pw"], scale=-2.0, x=x, normed_too=False)
    s = torch.empty(6, 520, dtype=torch.float32, device="cuda")
    got = om.block_norm(d["y"], weight=d["w"], sum_out=s, gate=d["r"])
    assert got[0] is s
    check(got, d["y"], w=d["w"], gate=d["r"], x=x, rx="f32")


@pytest.mark.parametrize("x", ["f16", "bf16"])
def test_weights_of_32_bits(x):
    d = inputs(5, 264, x, None, 9)
    w = {n: d[n].float() + 0.0001 for n in ("w", "b", "pw", "pb")}
    got = om.block_norm(d["y"], d["r"], w["w"], w["b"], post_weight=w["pw"], post_bias=w["pb"], norm="layer")
    check(got, d["y"], d["r"], w["w"], w["b"], w["pw"], w["pb"], kind="layer", x=x)


@pytest.mark.parametrize("x", ["f32", "f16"])
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 3), (2, 6), (4, 4), (8, 1)])
def test_strides_alignments_and_what_lies_beside_the_rows(x, shift, pad):
    tokens, width = 5, 328
    d = inputs(tokens, width, x, None, 21, "token")

    def wide(t):
        b = torch.full((tokens * (width + pad) + shift,), float("nan"), dtype=t.dtype, device="cuda")
        v = torch.as_strided(b, (tokens, width), (width + pad, 1), shift)
        v.copy_(t)
        return v, b

    y, r, g = (wide(d[n])[0] for n in ("y", "r", "gate"))
    (s, sb), (h, hb) = (wide(torch.zeros_like(d["y"])) for _ in range(2))
    got = om.block_norm(y, r, d["w"], post_weight=d["pw"], gate=g, activation="sigmoid", sum_out=s, out=h)
    assert got[0] is s and got[1] is h
    check(got, y, r, d["w"], pw=d["pw"], gate=g, act="sigmoid", x=x)
    for b in (sb, hb):  # nothing else was written
        assert int(torch.isnan(b).sum()) == b.numel() - tokens * width


def test_outputs_in_the_inputs_places():
    for rx in (None, "f32"):
        d = inputs(40, 512, "bf16", rx, 5, "channel")
        want = om.block_norm(d["y"], d["r"], d["w"], post_weight=d["pw"], gate=d["gate"], activation="silu")
        y, r = d["y"].clone(), d["r"].clone()
        got = om.block_norm(y, r, d["w"], post_weight=d["pw"], gate=d["gate"], activation="silu", sum_out=r, out=y)
        assert got[0] is r and got[1] is y and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    d = inputs(40, 512, "f32", None, 6)
    want = om.block_norm(d["y"], d["r"], d["w"])
    y, r = d["y"].clone(), d["r"].clone()
    got = om.block_norm(y, r, d["w"], sum_out=y, out=r)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(om.OmError):
        om.block_norm(y, r, d["w"], sum_out=y, out=y)


def test_one_row_for_all_tokens():
    d = inputs(33, 136, "bf16", None, 13)
    y, r = d["y"][:1].expand(33, 136), d["r"][:1].expand(33, 136)
    got = om.block_norm(y, r, d["w"], gate=d["gate"])
    want = om.block_norm(y.contiguous(), r.contiguous(), d["w"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_large_mean_costs_no_bits():
    """Rows of values near 4096 whose spread is 1: 12 bits of 24 are the mean's."""
    g = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randn(7, 5000, generator=g, device="cuda") + 4096.0
    check((None, om.block_norm(y, norm="layer")[1]), y, kind="layer")


def test_special_rows():
    d = inputs(8, 256, "f32", None, 17, "token")
    y, r, g = d["y"], d["r"], d["gate"]
    y[0, 3] = float("nan")
    y[1, 5] = float("inf")
    y[2] = 0.0
    r[2] = 0.0
    y[3] *= 1e-30
    r[3] *= 1e-30
    g[4] = float("-inf")
    g[5] = float("inf")
    g[6] = -200.0
    s, h = om.block_norm(y, r, d["w"], post_weight=d["pw"], gate=g, activation="silu")
    assert torch.isnan(s[0]).all() and torch.isnan(h[0]).all()
    assert torch.isnan(s[1, 5]) and torch.isnan(h[1]).all()
    assert torch.equal(s[2], torch.zeros_like(s[2])) and torch.equal(h[2], torch.zeros_like(h[2]))
    assert torch.equal(s[4], r[4])  # silu of minus infinity is 0
    assert not torch.isfinite(s[5]).any()
    assert torch.equal(s[6], r[6])
    rows = [3, 4, 6, 7]
    check((s[rows], h[rows]), y[rows], r[rows], d["w"], pw=d["pw"], gate=g[rows], act="silu")


def test_empty_calls():
    y = torch.empty(0, 64, device="cuda")
    s, h = om.block_norm(y, y, sum_out=None)
    assert s.shape == h.shape == (0, 64)
    y = torch.empty(3, 0, device="cuda")
    assert om.block_norm(y, y)[1].shape == (3, 0)


def test_binding_refuses():
    d = inputs(4, 64, "bf16", None, 2)
    y, r, w = d["y"], d["r"], d["w"]
    for bad in (dict(norm="batch"), dict(activation="relu", gate=r), dict(activation="silu"), dict(gate=r[:, :32]), dict(gate=w[:32]), dict(weight=w[:5]),
                dict(normed=False, weight=w), dict(residual=r[:3]), dict(out=torch.empty(4, 65, dtype=y.dtype, device="cuda"))):
        kw = dict(residual=r, weight=w)
        kw.update(bad)
        with pytest.raises(ValueError):
            om.block_norm(y, **kw)
    with pytest.raises(ValueError):
        om.block_norm(y, normed=False)
    for bad in (dict(residual=r.half()), dict(weight=w.half()), dict(bias=w.float()), dict(out=r.float()), dict(weight=w.cpu())):
        kw = dict(residual=r, weight=w)
        kw.update(bad)
        with pytest.raises(TypeError):
            om.block_norm(y, **kw)
    with pytest.raises(ValueError):
        om.block_norm(y.t().contiguous().t(), r, w)
    with pytest.raises(om.OmError):
        om.block_norm(torch.zeros(1, 40000, device="cuda"))


def test_on_another_stream_and_captured():
    d = inputs(64, 1024, "bf16", None, 8, "channel")
    want = om.block_norm(d["y"], d["r"], d["w"], gate=d["gate"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = om.block_norm(d["y"], d["r"], d["w"], gate=d["gate"], stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = om.block_norm(d["y"], d["r"], d["w"], gate=d["gate"])
    d["y"].mul_(0.5)
    graph.replay()
    want = om.block_norm(d["y"], d["r"], d["w"], gate=d["gate"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
