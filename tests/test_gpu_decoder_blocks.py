"""The attention layer with norms, a window with visible first tokens, several axes of positions and a
shared prefix: each is its operators one after the other, and its captured step the eager one."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


def layer_of(dtype=torch.bfloat16, codes=torch.int8, seqs=3, capacity=200, max_new=140, prefix=0, **kw):
    from implicit_gemm_convolution_gb300.decoder import AttentionLayer, LayerShape
    return AttentionLayer(LayerShape(model=320, q_heads=6, kv_heads=2, dim=64, rot=32, group=64, page=16, **kw), seqs, capacity, max_new, dtype=dtype, codes=codes,
                          prefix=prefix)


def prompt_of(layer, lens, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(sum(lens), layer.shape.model, generator=g, device="cuda").to(layer.dtype)
    counts = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return x, counts, torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def step_of(layer, seed=7):
    return torch.randn(layer.seqs, 320, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(layer.dtype)


NORMS = dict(norm="rms", post_norm=True, gate=True, residual_scale=0.5)
FULL = [dict(), NORMS, dict(norm="layer", window=30, sinks=3), dict(sections=(4, 6, 6)), dict(sections=(6, 5, 5), order="turns", **NORMS)]


@pytest.mark.parametrize("prefix", [0, 70])
@pytest.mark.parametrize("kw", FULL)
def test_a_layer_is_its_operators(kw, prefix):
    if prefix and kw.get("window"):
        pytest.skip("not together")
    layer, s = layer_of(prefix=prefix, **kw), layer_of(prefix=prefix, **kw).shape
    if prefix:
        layer.run_prefix(prompt_of(layer, [prefix], 2)[0])
    lens = [40, 7, 137]
    layer.run(*prompt_of(layer, lens))
    keep = [t.clone() for t in (layer.cache.k, layer.cache.v, layer.cache.k_scale, layer.cache.v_scale)]
    x = step_of(layer)
    y = layer.run(x)
    after = [t.clone() for t in (layer.cache.k, layer.cache.v, layer.cache.k_scale, layer.cache.v_scale)]
    for t, k in zip((layer.cache.k, layer.cache.v, layer.cache.k_scale, layer.cache.v_scale), keep):
        t.copy_(k)
    h = om.block_norm(x, weight=layer.norm_weight, norm=s.norm)[1] if s.norm else x
    rows = om.w4_matvec(h, *layer.qkv, group=64).view(3, 10, 64)
    places = torch.tensor([n + prefix for n in lens], dtype=torch.int32, device="cuda")
    q = om.kv_append(layer.cache, rows[:, :6], rows[:, 6:8], rows[:, 8:], layer.table, layer.block_table, layer.ctx_len, layer.one_each, 1,
                     positions=places.expand(3, -1).contiguous(), pair_axis=om.rope_axes(s.sections, s.order) if s.sections else None)
    assert all(torch.equal(a, b) for a, b in zip(after, (layer.cache.k, layer.cache.v, layer.cache.k_scale, layer.cache.v_scale)))
    if prefix:
        assert layer.prefix_len.tolist() == [prefix]
        o = om.kv_shared_attention(layer.cache, q, layer.prefix_table, layer.prefix_len, layer.groups, layer.block_table, layer.ctx_len, layer.one_each, 1)
    else:
        o = om.kv_attention(layer.cache, q, layer.block_table, layer.ctx_len, layer.one_each, 1, window=s.window, sinks=s.sinks, workspace=layer.workspace)
    o = om.w4_matvec(o.view(3, -1), *layer.out, group=64)
    if s.norm:
        want = om.block_norm(o, x, post_weight=layer.post_weight, gate=layer.gate, scale=s.residual_scale, norm=s.norm, normed=False)[0]
    else:
        want = o + x
    assert torch.equal(y, want) and torch.isfinite(y).all()


@pytest.mark.parametrize("prefix,kw", [(0, NORMS), (0, dict(window=30, sinks=3)), (0, dict(sections=(4, 6, 6))), (70, dict(sections=(4, 6, 6), **NORMS)), (70, dict())])
def test_a_captured_step_is_the_eager_step(prefix, kw):
    a, b = layer_of(prefix=prefix, **kw), layer_of(prefix=prefix, **kw)
    for l in (a, b):
        if prefix:
            l.run_prefix(prompt_of(l, [prefix], 2)[0])
        l.run(*prompt_of(l, [9, 40, 1]))
    x = step_of(a)
    graph, y = b.capture(x)
    for step in range(4):
        want = a.run(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), step
        assert torch.equal(a.cache.k, b.cache.k) and torch.equal(a.cache.v_scale, b.cache.v_scale)
        x.copy_(want)


def test_places_on_all_axes_are_the_places():
    a, b = layer_of(), layer_of(sections=(4, 6, 6))
    p = prompt_of(a, [9, 40, 1])
    assert torch.equal(a.run(*p), b.run(*p)) and torch.equal(a.run(step_of(a)), b.run(step_of(b)))
    c, d = layer_of(sections=(4, 6, 6)), layer_of(sections=(4, 6, 6))
    grid = torch.arange(50, dtype=torch.int32, device="cuda")
    positions = torch.stack((grid // 20, grid // 5 % 4, grid % 5))
    assert not torch.equal(c.run(*p), d.run(*p, positions=positions))


def test_a_shared_prefix_is_the_prefix_of_each(monkeypatch):
    """Against sequences that each hold the prefix themselves. The prefix fills its pages, so both caches hold the same codes, the queries are
    the same bits, and the attention's outputs differ by the two calls' own errors: a score (dim + 16) 2^-22 of its sum of magnitudes,
    twice that and 2^-18 of a weight."""
    from implicit_gemm_convolution_gb300 import decoder
    seen = []
    for name in ("kv_attention", "kv_shared_attention"):
        real = getattr(decoder, name)

        def spy(cache, q, *a, _real=real, **kw):
            out = _real(cache, q, *a, **kw)
            seen.append((q.clone(), out.clone()))
            return out
        monkeypatch.setattr(decoder, name, spy)
    prefix, lens = 64, [20, 7, 31]
    shared, alone = layer_of(torch.float32, prefix=prefix), layer_of(torch.float32, capacity=300)
    alone.qkv, alone.out = shared.qkv, shared.out
    head, tail = prompt_of(shared, [prefix], 2)[0], prompt_of(shared, lens)
    shared.run_prefix(head)
    shared.run(*tail)
    parts = [torch.cat((head, t)) for t in tail[0].split(lens)]
    each = [prefix + n for n in lens]
    counts = torch.tensor(each, dtype=torch.int32, device="cuda")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(each)]), dtype=torch.int32, device="cuda")
    alone.run(torch.cat(parts), counts, cu)
    step = step_of(shared)
    shared.run(step)
    alone.run(step)
    (q0, a0), (q1, a1), (q, a), (q2, a2), (q3, a3) = seen
    q, a = q.split(each), a.split(each)
    k, v = om.kv_read(alone.cache, alone.block_table, torch.zeros_like(counts), cu, 100, int(cu[-1]))
    heads = torch.arange(6, device="cuda") // 3
    for got, ours, theirs, want in [(q0, a0, q[0][:prefix], a[0][:prefix]), (q1, a1, torch.cat([x[prefix:] for x in q]), torch.cat([x[prefix:] for x in a])),
                                    (q2, a2, q3, a3)]:
        assert torch.equal(got, theirs)
        big = 64 ** -0.5 * torch.einsum("thd,phd->thp", got.abs(), k.abs()[:, heads]).amax(-1, keepdim=True)
        tol = 2 * (2 * 80 * 2.0 ** -22 * big + 2.0 ** -18) * v.abs()[:, heads].amax(0)
        assert bool(((ours - want).abs() <= tol).all()), float(((ours - want).abs() / tol).max())


def test_refusals():
    for kw in (dict(window=8, prefix=16), dict(post_norm=True), dict(gate=True), dict(residual_scale=0.5), dict(sections=(4, 4))):
        with pytest.raises(ValueError):
            layer_of(**kw)
    layer = layer_of(prefix=32)
    with pytest.raises(ValueError):
        layer.run_prefix(torch.zeros(33, 320, device="cuda").bfloat16())
