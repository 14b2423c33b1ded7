"""The decoding operators together: the attention half of a decoder layer over prompts and
steps, against 64 bits at every stage, and its step as a CUDA graph.

Each stage is compared with the 64-bit value of its own inputs (the rounded outputs of the stage before),
so the tolerances are the operators' own: 32-bit sums and one rounding to the type.
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


def small(dtype, codes, **kw):
    from implicit_gemm_convolution_gb300.decoder import AttentionLayer, LayerShape
    shape = LayerShape(model=320, q_heads=6, kv_heads=2, dim=64, rot=32, group=64, page=16)
    return AttentionLayer(shape, 3, 100, 40, dtype=dtype, codes=codes, **kw)


def prompt_of(layer, lens, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(sum(lens), layer.shape.model, generator=g, device="cuda").to(layer.dtype)
    counts = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    return x, counts, cu


@pytest.mark.parametrize("x,kind", [("f32", "int8"), ("bf16", "e4m3"), ("f16", "int8")])
def test_layer_against_64_bits(x, kind, monkeypatch):
    from implicit_gemm_convolution_gb300 import decoder
    seen = []
    for name in ("w4_matvec", "kv_append", "kv_attention"):
        real = getattr(decoder, name)

        def spy(*a, _real=real, _name=name, **kw):
            before = [t.clone() if isinstance(t, torch.Tensor) else t for t in a]
            out = _real(*a, **kw)
            seen.append((_name, before, out.clone()))
            return out
        monkeypatch.setattr(decoder, name, spy)
    layer = small(ref.TORCH[x], ref.CODE_DTYPE[kind])
    lens = [40, 7, 17]
    layer.run(*prompt_of(layer, lens))
    g = torch.Generator(device="cuda").manual_seed(6)
    ctx = np.array(lens)
    for step in range(4):
        seen.clear()
        xs = torch.randn(3, 320, generator=g, device="cuda").to(layer.dtype)
        y = layer.run(xs)
        ctx = ctx + 1
        assert layer.ctx_len.cpu().tolist() == ctx.tolist()
        assert [s[0] for s in seen] == ["w4_matvec", "kv_append", "kv_attention", "w4_matvec"]
        for i in (0, 3):
            a, w = seen[i][1][0], (layer.qkv, layer.out)[i == 3]
            W = ref.w4_weights(w[0], w[1], w[2], a.shape[1], 64)
            A = ref.f64(a)
            want, mag = A @ W.T, np.abs(A) @ np.abs(W).T
            assert (np.abs(ref.f64(seen[i][2]) - want) <= (a.shape[1] + 64) * 2.0 ** -23 * mag + 1.01 * ref.UNIT[x] * np.abs(want) + ref.TINY[x]).all()
        q = seen[1][2]
        out, _, mag, big = ref.attention(ref.f64(q), ref.code_values(layer.cache.k), ref.code_values(layer.cache.v), ref.f64(layer.cache.k_scale),
                                         ref.f64(layer.cache.v_scale), layer.block_table.cpu().numpy().astype(np.int64), ctx, np.arange(4), 64 ** -0.5, 0, 16)
        ew = 2 * (64 + 16) * 2.0 ** -22 * big + 2.0 ** -20 + (2.0 ** -20 if x == "f32" else 2.0 ** -10) + 100 * 2.0 ** -23
        assert (np.abs(ref.f64(seen[2][2]) - out) <= ew[..., None] * mag + 1.01 * ref.UNIT[x] * np.abs(out) + ref.TINY[x]).all()
        assert torch.equal(y, seen[3][2] + xs)


def test_the_cache_holds_the_prompt():
    """Keys read back are the rotated projections, within half a step of their page's scale."""
    layer = small(torch.float32, torch.int8)
    lens = [40, 7, 17]
    x, counts, cu = prompt_of(layer, lens)
    layer.run(x, counts, cu)
    fused = om.w4_matvec(x, *layer.qkv, group=64).view(-1, 10, 64)
    start = torch.zeros(3, dtype=torch.int32, device="cuda")
    k, v = om.kv_read(layer.cache, layer.block_table, start, cu, 40, sum(lens))
    pos = np.concatenate([np.arange(n) for n in lens])
    want_k = ref.rotate(fused[:, 6:8].cpu().numpy(), layer.table.cpu().numpy(), pos, 32, False)
    for got, want in ((k.cpu().numpy(), want_k), (v.cpu().numpy(), fused[:, 8:].cpu().numpy())):
        t = 0
        for b, n in enumerate(lens):
            for j in range(0, n, 16):
                part = slice(t + j, t + min(n, j + 16))
                step = np.abs(want[part]).max(axis=(0, 2)) / 127
                assert (np.abs(got[part] - want[part]).max(axis=(0, 2)) <= 0.5 * step * (1 + 1e-5)).all()
            t += n


def test_a_captured_step_is_the_eager_step():
    a, b = small(torch.bfloat16, torch.int8), small(torch.bfloat16, torch.int8)
    p = prompt_of(a, [9, 40, 1])
    a.run(*p)
    b.run(*p)
    x = torch.randn(3, 320, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    graph, y = b.capture(x)
    for step in range(5):
        want = a.run(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), step
        assert torch.equal(a.cache.k, b.cache.k) and torch.equal(a.cache.v_scale, b.cache.v_scale)
        x.copy_(want)
    assert b.ctx_len.cpu().tolist() == [14, 45, 6]


def test_quantize4_is_within_half_a_step():
    from implicit_gemm_convolution_gb300.decoder import quantize4
    w = torch.randn(20, 131, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    w[3] = 0.0
    w[4] = w[4].abs()
    codes, scale, zero = quantize4(w, 64)
    back = ref.w4_weights(codes, scale, zero, 131, 64)
    step = ref.f64(scale)[:, np.arange(131) // 64]
    # the zero point is rounded too: a value at the end of its range can be a whole half step further
    assert (np.abs(back - ref.f64(w)) <= 1.0 * step * (1 + 1e-5) + 1e-7).all()
