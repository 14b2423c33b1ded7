"""The decoding operators' binding and the devices of its tensors, on the host: stand-ins say which device they are on."""
from contextlib import contextmanager

import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from implicit_gemm_convolution_gb300 import decode  # noqa: E402


class On(torch.Tensor):
    """A tensor that says it is on CUDA device `at`."""

    is_cuda = True

    def get_device(self):
        return self.at


def on(at, t):
    t = torch.Tensor._make_subclass(On, t)
    t.at = at
    return t


def operands(at, **other):
    """Operands of every operator on device `at`, those named in `other` on another."""
    make = dict(x=torch.zeros(2, 64), weight=torch.zeros(8, 32, dtype=torch.uint8), scales=torch.zeros(8, 2), zeros=torch.zeros(8, 2, dtype=torch.uint8),
                out=torch.zeros(2, 8), k=torch.zeros(3, 2, 64), v=torch.zeros(3, 2, 64), q=torch.zeros(3, 4, 64), q_out=torch.zeros(3, 4, 64),
                table=torch.zeros(9, 8, 2), block_table=torch.zeros(2, 4, dtype=torch.int32), ctx_len=torch.zeros(2, dtype=torch.int32),
                cu=torch.zeros(3, dtype=torch.int32), o=torch.zeros(3, 4, 64), lse=torch.zeros(3, 4), workspace=torch.zeros(1 << 20),
                k_out=torch.zeros(3, 2, 64), v_out=torch.zeros(3, 2, 64), codes=torch.zeros(5, 2, 16, 64, dtype=torch.int8), values=torch.zeros(5, 2, 16, 64, dtype=torch.int8),
                k_scale=torch.zeros(5, 2), v_scale=torch.zeros(5, 2))
    return {n: on(other.get(n, at), t) for n, t in make.items()}


def calls(t, stream=None):
    """(the names of its tensors, the call) of each operator."""
    cache = lambda: om.PagedKVCache(t["codes"], t["values"], t["k_scale"], t["v_scale"])
    in_cache, batch = ["codes", "values", "k_scale", "v_scale"], ["block_table", "ctx_len", "cu"]
    return {
        "om_w4_matvec": (["x", "weight", "scales", "zeros", "out"],
                         lambda: om.w4_matvec(t["x"], t["weight"], t["scales"], zeros=t["zeros"], group=32, out=t["out"], stream=stream)),
        "om_kv_append": (in_cache + batch + ["q", "k", "v", "table", "q_out"],
                         lambda: om.kv_append(cache(), t["q"], t["k"], t["v"], t["table"], t["block_table"], t["ctx_len"], t["cu"], 2, q_out=t["q_out"], stream=stream)),
        "om_kv_read": (in_cache + batch + ["k_out", "v_out"],
                       lambda: om.kv_read(cache(), t["block_table"], t["ctx_len"], t["cu"], 2, 3, k_out=t["k_out"], v_out=t["v_out"], stream=stream)),
        "om_kv_attention": (in_cache + batch + ["q", "o", "lse", "workspace"],
                            lambda: om.kv_attention(cache(), t["q"], t["block_table"], t["ctx_len"], t["cu"], 2, out=t["o"], lse=t["lse"], workspace=t["workspace"], stream=stream)),
    }


OPERATORS = ["om_w4_matvec", "om_kv_append", "om_kv_read", "om_kv_attention"]


@pytest.fixture
def seen(monkeypatch):
    """What reaches the library: (function, current device, stream). Device 0 is current; the current stream of device d is 1000 + d."""
    seen, current = [], [0]

    @contextmanager
    def device(d):
        was, current[0] = current[0], d
        yield
        current[0] = was

    class Library:
        def __getattr__(self, name):
            return lambda *args: seen.append((name, current[0], args[-1])) or 0

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    monkeypatch.setattr(decode, "_functions", Library())
    return seen


@pytest.mark.parametrize("name", OPERATORS)
def test_tensors_on_different_devices_are_refused(name, seen):
    tensors = calls(operands(0))[name][0]
    calls(operands(0))[name][1]()
    for t in tensors:
        with pytest.raises(ValueError):
            calls(operands(0, **{t: 1}))[name][1]()
    assert len(seen) == 1


@pytest.mark.parametrize("name", OPERATORS)
def test_calls_run_on_their_tensors_device(name, seen):
    for d in (0, 1):
        calls(operands(d))[name][1]()
    assert seen == [(name, 0, 1000), (name, 1, 1001)] and torch._C._cuda_getDevice() == 0


@pytest.mark.parametrize("name", OPERATORS)
def test_streams_of_another_device_are_refused(name, seen):
    class Stream:
        device_index, cuda_stream = 1, 77

    calls(operands(1), Stream())[name][1]()
    with pytest.raises(ValueError):
        calls(operands(0), Stream())[name][1]()
    assert seen == [(name, 1, 77)]
