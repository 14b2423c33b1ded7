"""The attention layer on a batch padded with rows that no sequence owns, and on a prefix of the most tokens it was made for."""
import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests.test_gpu_decoder_blocks import NORMS, layer_of, prompt_of, step_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


@pytest.mark.parametrize("prefix,kw", [(0, dict()), (0, dict(sections=(4, 6, 6), **NORMS)), (70, dict()), (70, dict(sections=(6, 5, 5), order="turns"))])
def test_rows_behind_the_last_sequence(prefix, kw):
    a, b = layer_of(prefix=prefix, **kw), layer_of(prefix=prefix, **kw)
    x, counts, cu = prompt_of(a, [40, 7, 90])
    for l in (a, b):
        if prefix:
            l.run_prefix(prompt_of(l, [prefix], 2)[0])
    want = a.run(x, counts, cu)
    got = b.run(torch.cat((x, torch.full_like(x[:23], 3.0))), counts, cu)
    assert torch.equal(got[:137], want) and torch.isfinite(want).all()
    assert torch.equal(a.cache.k, b.cache.k) and torch.equal(a.cache.v_scale, b.cache.v_scale) and torch.equal(a.ctx_len, b.ctx_len)
    assert torch.equal(a.run(step_of(a)), b.run(step_of(b)))
