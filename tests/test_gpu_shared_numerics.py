"""Attention of sequences that share prefixes: the order of its products, and bounds of its sums."""
import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests import decode_ref as ref  # noqa: E402
from tests.test_gpu_shared_attention import Shared, long_parts  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scores_leave_weights_that_are_still_read(dim, x):
    """A tile's scores take the columns of the weights of the tile before the last. Queries are zero, so a score is the bits of a
    weight 0, and values are all the same: a weight that its product has not read yet is missing from the output, at least one in 3000
    of the sum. Otherwise the weighted mean is the value to some units of 32 bits (weights and sums are whole numbers times one
    factor), and half a unit of the output's type. Another stream's work moves the tiles' times."""
    s = Shared([3000, 1300], [0, 40, 70], [3] * 70, [1] * 70, 4, dim, 64, "int8", 9)
    s.v = torch.full_like(s.v, 100)
    s.vs[:] = 0.0123
    s.device()
    q = torch.zeros(70, 32, dim, device="cuda").to(ref.TORCH[x])
    want = 100 * float(torch.tensor(0.0123))
    ws, side = s.workspace(32), torch.cuda.Stream()
    a = torch.randn(2048, 2048, device="cuda").bfloat16()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for i in range(12):
        with torch.cuda.stream(side):
            for _ in range(i):
                a @ a
        outs.append(s.attend(q, workspace=ws))
    torch.cuda.synchronize()
    assert om.workspace_status(ws) == 0
    for out in outs:
        assert torch.equal(out, outs[0])
    # cut sums: as far as the fold (32-bit queries) or the whole prefix goes
    tol = {"f32": 2.0 ** -18, "f16": 2.0 ** -15 + ref.UNIT["f16"], "bf16": 2.0 ** -15 + ref.UNIT["bf16"]}[x]
    assert float((outs[0].double() - want).abs().max()) <= tol * want


def one_token_each(prefix, seqs, hq, dim, page, kind, seed):
    """Sequences of one token of their own behind one prefix, one key head."""
    return Shared([prefix], [0, seqs], [1] * seqs, [1] * seqs, 1, dim, page, kind, seed, extra=0)


def against_64_bits(s, q, x):
    """check() of test_gpu_shared_attention.py on the device, with its tolerance, for one_token_each."""
    prefix, (tokens, hq, dim), scale = s.prefixes[0], q.shape, s.dim ** -0.5
    s.device()
    ws, lse = s.workspace(hq), torch.empty(tokens, hq, device="cuda")
    out = s.attend(q, lse=lse, workspace=ws)
    assert om.workspace_status(ws) == 0
    assert torch.equal(s.attend(q, workspace=ws), out)
    pos = torch.arange(prefix, device="cuda")
    ids, rows = torch.from_numpy(s.ptable_np[0]).cuda()[pos // s.page], pos % s.page
    own = torch.from_numpy(s.table_np[:, 0]).cuda()
    k, v = (c.float()[ids, 0, rows].double() * t[ids, 0][:, None].double() for c, t in ((s.k, s.ks), (s.v, s.vs)))
    ko, vo = (c.float()[own, 0, 0].double() * t[own, 0][:, None].double() for c, t in ((s.k, s.ks), (s.v, s.vs)))
    qq = q.double()
    y = scale * torch.cat((torch.einsum("thd,ld->thl", qq, k), torch.einsum("thd,td->th", qq, ko)[..., None]), -1)
    big = scale * torch.cat((torch.einsum("thd,ld->thl", qq.abs(), k.abs()), torch.einsum("thd,td->th", qq.abs(), ko.abs())[..., None]), -1).amax(-1)
    total = torch.logsumexp(y, -1)
    w = (y - total[..., None]).exp()
    mix = lambda a, b: w[..., :-1] @ a + w[..., -1:] * b[:, None]
    want, mag = mix(v, vo), mix(v.abs(), vo.abs())
    steps = prefix / 8 + 64
    ds = (dim + 16) * 2.0 ** -22 * big
    tol = (2 * ds + 2.0 ** -19 + steps * 2.0 ** -22)[..., None] * mag + 1.01 * ref.UNIT[x] * want.abs() + ref.TINY[x] + 1e-30
    off = (out.double() - want).abs()
    assert bool((off <= tol).all()), f"outputs {float((off / tol).max())} of the tolerance"
    assert bool(((lse.double() - total).abs() <= ds + (steps + 64) * 2.0 ** -22 + 2.0 ** -20 + 2.0 ** -22 * total.abs()).all()), "lse"


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("far", [1, 7, 8, 9, 20, 40, 90])
@pytest.mark.parametrize("page,dim", [(16, 64), (32, 128), (16, 256), (64, 128)])
def test_scales_far_apart_in_one_tile(page, dim, far, kind, x):
    """Pages of one tile whose tokens weigh about the same, their value scales 2^far apart. In odd dimensions the pages of the large scale
    hold zeros, so what comes out there is the others', to the precision that they would have alone."""
    s = one_token_each(333, 5, 8, dim, page, kind, far + page)
    large = torch.arange(s.pages, device="cuda") % 2 == 0
    g = torch.Generator(device="cuda").manual_seed(far)
    s.vs[:, 0] = torch.where(large, 1.0, 2.0 ** -far) * (0.5 + torch.rand(s.pages, generator=g, device="cuda"))
    odd = torch.arange(dim, device="cuda") % 2 == 1
    s.v.view(torch.int8)[large[:, None, None, None] & odd[None, None, None, :].expand(s.v.shape[0], 1, page, dim)] = 0
    s.vs[torch.from_numpy(s.table_np[:, 0]).cuda()] = 2.0 ** -far  # the own tokens: as small
    s.v.view(torch.int8)[torch.from_numpy(s.table_np[:, 0]).cuda()] = 0
    q = 0.1 * torch.randn(5, 8, dim, generator=g, device="cuda")
    against_64_bits(s, q.to(ref.TORCH[x]), x)
    against_64_bits(s, torch.zeros_like(q).to(ref.TORCH[x]), x)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("page,dim,prefix", [(16, 64, 16003), (32, 128, 9000), (16, 256, 5000)])
def test_scales_of_all_sizes_over_long_parts(page, dim, prefix, kind, x):
    """Several tiles a block (sums of 32-bit queries leave tensor memory among them), value scales of every page anywhere in 2^50, some 0 or
    negative, large ones with zeros in odd dimensions; maxima that rise towards the end."""
    s = one_token_each(prefix, 260, 10, dim, page, kind, prefix)
    g = torch.Generator(device="cuda").manual_seed(3)
    power = torch.randint(-45, 6, (s.pages,), generator=g, device="cuda")
    sign = torch.randint(-1, 2, (s.pages,), generator=g, device="cuda") | 1
    s.vs[:, 0] = torch.exp2(power.float()) * sign * (torch.rand(s.pages, generator=g, device="cuda") > 0.05)
    odd = torch.arange(dim, device="cuda") % 2 == 1
    s.v.view(torch.int8)[(power > -20)[:, None, None, None] & odd[None, None, None, :].expand(s.v.shape[0], 1, page, dim)] = 0
    pages = torch.from_numpy(s.ptable_np[0]).cuda()[: -(-prefix // page)]
    s.ks[pages, 0] = torch.linspace(1e-5, 1e-2, len(pages), device="cuda")
    q = torch.randn(260, 10, dim, generator=g, device="cuda")
    against_64_bits(s, q.to(ref.TORCH[x]), x)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_sums_of_one_sign_are_cut_for_four_tiles_only(dim):
    """32-bit queries of zero behind 131072 tokens: weights are equal, values of one sign, so what the tensor cores cut off adds up. A step of 16
    positions and one of two parts cuts at most a unit in the last place of the sum so far, 2^-23 of it: 32 steps in four tiles, on
    average half of the sum, 16.5 of them. Then each fold rounds half a unit of the sum so far, half of the part's on average; the rest
    (weights in two parts, means, the join of some ten parts) is 2^-21. Sums that stayed for 16 tiles would be 66 units off."""
    worst = long_parts("f32", dim, 512, 8, 131072, 600, True, 50)
    blocks = torch.cuda.get_device_properties(0).multi_processor_count * (1 if dim == 256 else 2)
    tiles = -(-(131072 // 64) * (512 * 8 // 128) // blocks)  # of a block
    assert worst <= 16.5 * 2.0 ** -23 + tiles / 4 / 2 * 2.0 ** -24 + 2.0 ** -21, worst


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_what_is_not_finite_beside_scales_far_apart(x):
    """Tiles that come again: NaN codes behind the prefix's end and pages that are not there stay hidden in every pass, a scale or a visible code that
    is NaN shows."""
    s = Shared([200, 200], [0, 2, 4], [1] * 4, [1] * 4, 1, 64, 16, "e4m3", 5, extra=0)
    first, last = s.ptable_np[0], s.ptable_np[1]
    s.vs[torch.from_numpy(first[::2].copy()).cuda()] *= 2.0 ** -40
    s.vs[torch.from_numpy(last[1::2].copy()).cuda()] *= 2.0 ** -60
    for t in (s.k, s.v):
        t.view(torch.int8)[int(first[12]), :, 8:] = 0x7F  # positions 200 .. 207 of the first prefix
    s.ptable_np[0, 3] = -1
    s.device()
    q = torch.randn(4, 8, 64, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(ref.TORCH[x])
    ws = s.workspace(8)
    out = s.attend(q, workspace=ws)
    assert torch.isfinite(out).all()
    for change in (lambda: s.vs.__setitem__((int(last[4]), 0), float("inf")), lambda: s.ks.__setitem__((int(last[7]), 0), float("nan")),
                   lambda: s.v.view(torch.int8).__setitem__((int(last[5]), 0, 3), 0x7F)):
        keep = [t.view(torch.int8).clone() if t.element_size() == 1 else t.clone() for t in (s.vs, s.ks, s.v)]
        change()
        got = s.attend(q, workspace=ws)
        assert torch.equal(got[:2], out[:2]) and torch.isnan(got[2:]).all()
        for t, k in zip((s.vs, s.ks, s.v), keep):
            (t.view(torch.int8) if t.element_size() == 1 else t).copy_(k)
    assert torch.equal(s.attend(q, workspace=ws), out) and om.workspace_status(ws) == 0
