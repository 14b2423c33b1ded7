"""The decoding operators on streams other than the current one."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests.test_gpu_decode import Batch, gen, w4_inputs  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


def w4_call():
    X, U, S, Z = w4_inputs(16, 40000, 64, 32, "f32", True, 5)
    return lambda stream: om.w4_matvec(X, U, S, zeros=Z, group=32, stream=stream)


def batch_calls():
    bt = Batch([600, 600], [600, 600], 8, 128, 64, "int8", 4).device()
    q = torch.randn(1200, 8, 128, generator=gen(1), device="cuda")
    return bt, q


CALLS = ["w4_matvec", "kv_append", "kv_read", "kv_attention"]


def call_of(name):
    """A function of the stream that returns the outputs which the call allocates."""
    if name == "w4_matvec":
        return w4_call()
    bt, q = batch_calls()
    if name == "kv_append":
        table = om.rope_table(700, 128)
        return lambda stream: om.kv_append(bt.cache, q, q, q, table, bt.table, bt.lens, bt.cu, 600, stream=stream)
    if name == "kv_read":
        start = torch.zeros(2, dtype=torch.int32, device="cuda")
        return lambda stream: om.kv_read(bt.cache, bt.table, start, bt.cu, 600, 1200, stream=stream)
    return lambda stream: om.kv_attention(bt.cache, q, bt.table, bt.lens, bt.cu, 600, stream=stream)


@pytest.mark.parametrize("name", CALLS)
def test_outputs_of_a_call_on_another_stream_do_not_take_memory_in_use(name):
    """A tensor is freed while the current stream still has to read it: a call on another stream takes other memory."""
    call = call_of(name)
    want = call(None)
    many = isinstance(want, tuple)
    first = want[0] if many else want
    want = [t.clone() for t in (want if many else (want,))]
    shape = first.shape
    side = torch.cuda.Stream()
    call(side)  # loaded before what follows
    del first
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full(shape, 5.0, device="cuda") for _ in range(2)]
    copies = [torch.empty_like(t) for t in held]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for c, t in zip(copies, held):
        c.copy_(t)
    held.clear()
    del t
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all((c == 5.0).all() for c in copies)
    for g, w in zip(got if many else (got,), want):
        assert torch.equal(g, w)
