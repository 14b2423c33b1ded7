"""Attention: windows as long as their type can hold, and tokens that no sequence owns."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests.test_gpu_decode import Batch, gen  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


@pytest.mark.parametrize("window", [2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 62, 2 ** 63 - 8, 2 ** 63 - 1])
def test_a_window_longer_than_any_sequence_is_none(window):
    """Sequences with more queries than tokens among them: their first positions are negative, and less the window below 64 bits."""
    bt = Batch([2, 100, 0, 7, 300], [9, 3, 4, 7, 1], 2, 64, 16, "int8", 4).device()
    q = torch.randn(24, 8, 64, generator=gen(1), device="cuda")
    got, want = torch.empty(24, 8, device="cuda"), torch.empty(24, 8, device="cuda")
    a = om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, 9, window=window, lse=got)
    b = om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, 9, lse=want)
    assert torch.equal(a, b) and torch.equal(got, want)


@pytest.mark.parametrize("x", [torch.float32, torch.bfloat16])
def test_rows_that_no_sequence_owns_stay(x):
    bt = Batch([30, 90], [3, 2], 2, 64, 16, "int8", 6).device()
    q = torch.randn(11, 8, 64, generator=gen(1), device="cuda").to(x)
    out, lse = torch.full_like(q, 7.0), torch.full((11, 8), 7.0, device="cuda")
    om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, 3, out=out, lse=lse, workspace=om.new_kv_workspace(bt.cache, 8, 3))
    want = om.kv_attention(bt.cache, q[:5].contiguous(), bt.table, bt.lens, bt.cu, 3)
    assert torch.equal(out[:5], want) and (out[5:] == 7).all() and (lse[5:] == 7).all() and (lse[:5] != 7).all()
