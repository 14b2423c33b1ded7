"""Attention of sequences that share prefixes: the order of its products, and bounds of its sums."""
import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests import decode_ref as ref  # noqa: E402
from tests.test_gpu_shared_attention import Shared  # noqa: E402

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
