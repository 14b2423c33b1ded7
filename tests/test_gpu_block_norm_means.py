"""Layer norms of rows whose mean is large, and gates far out, against the formula in 64 bits.

Tolerances, u = 2^-24, as in test_gpu_block_norm.py: a sum of one sign is off by 43 u of itself, 64 u with its division. A 32-bit value less
a mean near it is exact, so what the first mean is off by (64 u of the mean magnitude at most) is in every difference alike and comes out
with the differences' own mean, which is off by 64 u of their mean magnitude. After that the row is one of mean 0.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import implicit_gemm_convolution_gb300 as om  # noqa: E402
from tests import decode_ref as ref  # noqa: E402
from tests.test_gpu_block_norm import U, normed  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    om.build()
    om.lib()


def layer_normed(y, w=None, b=None, eps=1e-6):
    v = ref.f64(y)
    c = v - v.mean(-1, keepdims=True)
    first = 64 * U * np.abs(v).mean(-1, keepdims=True)
    tol = 64 * U * (np.abs(c).mean(-1, keepdims=True) + first) + U * np.abs(c)
    return normed(c, tol, "rms", None if w is None else ref.f64(w), None if b is None else ref.f64(b), float(np.float32(eps)))


@pytest.mark.parametrize("mean,spread", [(4096.0, 1.0), (-300.0, 0.01), (0.0, 1.0), (1e6, 30.0)])
@pytest.mark.parametrize("tokens,width", [(5, 64), (9, 1000), (700, 300), (7, 5000), (310, 4096), (3, 8177), (4, 16383), (3, 32767), (4, 32768)])
def test_a_large_mean_costs_no_bits(tokens, width, mean, spread):
    g = torch.Generator(device="cuda").manual_seed(width)
    y = torch.randn(tokens, width, generator=g, device="cuda") * spread + mean
    w, b = torch.randn(width, generator=g, device="cuda"), torch.randn(width, generator=g, device="cuda")
    want, tol = layer_normed(y, w, b)
    off = np.abs(ref.f64(om.block_norm(y, weight=w, bias=b, norm="layer")[1]) - want)
    tol = tol + ref.UNIT["f32"] * np.abs(want)
    assert (off <= tol).all(), f"{float((off / tol).max())} of the tolerance"
    # before the residual, too
    x = om.block_norm(y, torch.zeros_like(y), post=True, norm="layer", normed=False)[0]
    want, tol = layer_normed(y)
    off = np.abs(ref.f64(x) - want)
    tol = tol + 2 * U * np.abs(want)
    assert (off <= tol).all(), f"{float((off / tol).max())} of the tolerance"


@pytest.mark.parametrize("width", [64, 1000, 8177])
def test_rows_of_one_value(width):
    """The variance is 0: what is left is rounding, far below sqrt(eps), and no root of a negative number."""
    y = torch.tensor([[4096.3], [-1e-3], [0.0], [7.1e5]], device="cuda").expand(4, width).contiguous()
    h = om.block_norm(y, norm="layer", eps=1e-6)[1]
    # differences are at most 64 u of the value before their mean is taken out, 65 u of that after
    tol = 66 * U * 64 * U * np.abs(ref.f64(y)) * 1e3 + 1e-37
    assert (np.abs(ref.f64(h)) <= tol).all()


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("width", [64, 1000, 4096])
def test_a_gate_that_is_shut(act, width):
    """Gates of minus infinity and far below 0 let nothing through, however large the block's output is; the sigmoid is e^-g below
    about 2^-125, where the factor counts as 0."""
    gates = [float("-inf"), -1e4, -200.0, -89.0, -86.0, 0.0, 200.0]
    y = torch.full((len(gates), width), 1e30, device="cuda")
    g = torch.tensor(gates, device="cuda")[:, None].expand(-1, width).contiguous()
    x = om.block_norm(y, torch.zeros_like(y), gate=g, activation=act, normed=False)[0]
    assert (x[:4] == 0).all()
    v = ref.f64(g[4:])
    want = 1e30 / (1 + np.exp(-v)) * (v if act == "silu" else 1.0)
    assert (np.abs(ref.f64(x[4:]) - want) <= 10 * U * np.abs(want)).all()
