"""The attention layer's count of its tokens' places, which needs no GPU."""
import pytest

torch = pytest.importorskip("torch")

from implicit_gemm_convolution_gb300.decoder import places  # noqa: E402


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


@pytest.mark.parametrize("ctx,new", [([5], [5]), ([9, 4, 30], [1, 1, 1]), ([3, 8, 8, 2, 7], [3, 0, 4, 0, 7]), ([6, 5], [0, 2]), ([4, 6], [0, 0])])
@pytest.mark.parametrize("padded", [0, 1, 9])
def test_places_of_batches(ctx, new, padded):
    """Sequences without new tokens among them; a batch padded with rows that no sequence owns, which the operators leave alone."""
    cu = [sum(new[:b]) for b in range(len(new) + 1)]
    got = places(i32(ctx), i32(cu), cu[-1] + padded)
    assert got.dtype == torch.int32 and got.shape == (cu[-1] + padded,)
    assert got[:cu[-1]].tolist() == [c - n + i for c, n in zip(ctx, new) for i in range(n)]
