"""Capturing a step of the attention layer leaves what the layer holds as it is."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests.test_gpu_decoder import prompt_of, small  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


def held(layer):
    c = layer.cache
    return [t.view(torch.int8).clone() if t.element_size() == 1 else t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale, layer.ctx_len, layer.block_table)]


@pytest.mark.parametrize("placeholder", [50.0, float("nan"), float("inf")])
@pytest.mark.parametrize("kind", [torch.int8, torch.float8_e4m3fn])
def test_capture_on_a_buffer_that_is_not_filled(kind, placeholder):
    """Pages that are partly full: what the buffer holds at the capture changes neither their scales nor their codes."""
    a, b = small(torch.bfloat16, kind), small(torch.bfloat16, kind)
    p = prompt_of(a, [9, 40, 1])
    a.run(*p)
    b.run(*p)
    before = held(b)
    x = torch.full((3, 320), placeholder, device="cuda").bfloat16()
    graph, y = b.capture(x)
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(before, held(b)))
    x.copy_(torch.randn(3, 320, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda"))
    for step in range(3):
        want = a.run(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(y).all() and torch.equal(y, want), step
        assert all(torch.equal(s, t) for s, t in zip(held(a), held(b))), step
        x.copy_(want)
