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


def test_the_longest_prefix_and_the_longest_sequence_behind_it():
    """A prefix that ends inside a page: the sequence's last token is at the table's last row. One token more is refused, where it had been
    taken into the page's room and the last own tokens came out NaN."""
    layer = layer_of(prefix=40, capacity=20, max_new=20)
    with pytest.raises(ValueError):
        layer.run_prefix(prompt_of(layer, [41], 2)[0])
    assert layer.prefix_len.tolist() == [0]
    layer.run_prefix(prompt_of(layer, [40], 2)[0])
    layer.run(*prompt_of(layer, [19, 3, 19]))
    assert torch.isfinite(layer.run(step_of(layer))).all() and layer.ctx_len.tolist() == [20, 4, 20]
