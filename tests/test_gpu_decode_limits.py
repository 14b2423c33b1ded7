"""The decoding operators at the ends of their operands and ranges."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests import decode_ref as ref  # noqa: E402
from tests.test_gpu_decode import Batch, attend_and_check, check_w4, gen, i32, w4_inputs  # noqa: E402


@pytest.mark.parametrize("n", [33, 34, 35, 36])
@pytest.mark.parametrize("at", [0, 1, 2, 3])
def test_w4_zero_points_to_their_last_byte(n, at):
    """Two groups a row: the rows behind the last whole tile are fewer bytes than a copy."""
    k, group = 256, 128
    X, U, S, Z = w4_inputs(2, n, k, group, "bf16", True, n + at)
    flat = torch.full((at + 2 * n,), 255, dtype=torch.uint8, device="cuda")
    z = flat[at:].view(n, 2)
    z.copy_(Z)
    check_w4(om.w4_matvec(X, U, S, zeros=z, group=group), X, U, S, Z, k, group, "bf16")
