"""The decoding operators on another device than the process's first."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import implicit_gemm_convolution_gb300 as om  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_a_layer_on_each_device():
    """What is set up for a kernel on one device is not taken for set up on the other."""
    from implicit_gemm_convolution_gb300.decoder import AttentionLayer, LayerShape
    for device in (0, 1):
        with torch.cuda.device(device):
            layer = AttentionLayer(LayerShape(model=2048, page=16), 2, 200, 8)
            x = torch.randn(2, 2048, device="cuda").bfloat16()
            for _ in range(3):
                x = layer.run(x)
            assert torch.isfinite(x).all()


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_a_layer_on_a_device_that_is_not_the_current_one():
    from implicit_gemm_convolution_gb300.decoder import AttentionLayer, LayerShape
    layer = AttentionLayer(LayerShape(model=2048, page=16), 2, 200, 8, device="cuda:1")
    x = torch.randn(2, 2048, device="cuda:1").bfloat16()
    for _ in range(3):
        x = layer.run(x)
    assert torch.isfinite(x).all()
    with pytest.raises(ValueError):
        om.w4_matvec(torch.zeros(2, 2048, device="cuda:0").bfloat16(), *layer.qkv, group=128)
