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


def test_attention_offsets_that_decrease_are_bounded():
    """Every second sequence claims the whole batch: their units together pass 32 bits, so nothing is done."""
    seqs, tokens, page, width = 4096, 2048, 128, 512
    bt = Batch([page], [1], 8, 64, page, "int8", 3).device()
    q = torch.ones(tokens, 32, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, -7.0)
    cu = i32([0, tokens] * (seqs // 2) + [0])
    table = torch.zeros(seqs, width, dtype=torch.int32, device="cuda")
    ctx = torch.full((seqs,), page * width, dtype=torch.int32, device="cuda")
    ws = om.new_kv_workspace(bt.cache, 32, tokens)
    om.kv_attention(bt.cache, q, table, ctx, cu, tokens, out=out, workspace=ws)
    assert (out == -7).all() and om.device_status() == 0


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("x,kind,dim,hq", [("f32", "int8", 128, 4), ("bf16", "e4m3", 128, 8), ("bf16", "int8", 64, 20), ("f32", "e4m3", 256, 2)])
def test_attention_values_near_the_end_of_the_range(x, kind, dim, hq, workspace):
    """Means of thousands of values near 1e36: their plain sums have no 32-bit float."""
    bt = Batch([5000, 700], [1, 1], 2, dim, 64, kind, dim + hq)
    bt.vs = bt.vs * 1e36
    attend_and_check(bt, hq, x, workspace=workspace)
