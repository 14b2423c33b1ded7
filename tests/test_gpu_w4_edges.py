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
