"""The 4-bit product at sizes and values beside the usual ones."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests import decode_ref as ref  # noqa: E402
from tests.test_gpu_decode import check_w4, w4_inputs  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


@pytest.mark.parametrize("x,m,n,k,group,zeros", [
    ("bf16", 1, 50257, 96, 32, True), ("f32", 2, 128256, 64, 64, False), ("f16", 16, 40001, 520, 128, True), ("f32", 7, 39000, 1300, 128, False),
])
def test_more_rows_than_one_pass(x, m, n, k, group, zeros):
    """Vocabulary projections: a block runs its tiles in several passes."""
    X, U, S, Z = w4_inputs(m, n, k, group, x, zeros, n)
    check_w4(om.w4_matvec(X, U, S, zeros=Z, group=group), X, U, S, Z, k, group, x)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("group,k", [(384, 384), (384, 1200), (640, 1281), (1152, 4096), (256, 300)])
def test_wide_groups(group, k, x):
    for m, zeros in ((1, True), (9, False)):
        X, U, S, Z = w4_inputs(m, 70, k, group, x, zeros, k)
        check_w4(om.w4_matvec(X, U, S, zeros=Z, group=group), X, U, S, Z, k, group, x)


@pytest.mark.parametrize("group,k", [(256, 2000), (1024, 2048), (384, 1153)])
@pytest.mark.parametrize("at", [0, 1, 2, 3])
def test_wide_groups_from_the_operands_first_byte(at, group, k):
    """Scales and zero points that begin inside a word: the first rows' groups go on in units behind the first."""
    n, groups = 40, -(-k // group)
    X, U, S, Z = w4_inputs(3, n, k, group, "bf16", True, at)
    z = torch.full((at + n * groups,), 255, dtype=torch.uint8, device="cuda")[at:].view(n, groups)
    s = torch.full((at + n * groups,), float("nan"), dtype=S.dtype, device="cuda")[at:].view(n, groups)
    z.copy_(Z)
    s.copy_(S)
    check_w4(om.w4_matvec(X, U, s, zeros=z, group=group), X, U, S, Z, k, group, "bf16")


@pytest.mark.parametrize("x", ["f16", "bf16"])
@pytest.mark.parametrize("m", [4, 11])
def test_16_bit_activations_that_are_not_finite(x, m):
    """Infinities and NaN reach exactly the rows that hold them."""
    n, k, group = 50, 300, 64
    X, U, S, Z = w4_inputs(m, n, k, group, x, False, m)
    U[:, 0] = 0x1F  # codes 15 and 1: neither is the zero point
    X[1, 0] = float("inf")
    X[2, 1] = float("inf")
    X[3, 1] = float("nan")
    y = om.w4_matvec(X, U, S, group=group)
    assert torch.isinf(y[1]).all() and (y[1] > 0).all() and torch.isinf(y[2]).all() and (y[2] < 0).all() and torch.isnan(y[3]).all()
    rows = [0] + list(range(4, m))
    check_w4(y[rows], X[rows], U, S, Z, k, group, x)
