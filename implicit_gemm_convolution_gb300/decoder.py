"""The attention half of a decoder layer on the decoding operators: 4-bit products,
the append to a paged 8-bit cache with the position rotation, and attention over it.

One call of :meth:`AttentionLayer.run` takes any number of new tokens of each sequence: a
prompt, or one token of every sequence (:meth:`AttentionLayer.capture` makes a CUDA
graph of that step; lengths live on the device and grow with every replay). The
operators are the library's; what is torch here is bookkeeping (slicing the fused
projection, adding the residual, counting positions).

``python -m implicit_gemm_convolution_gb300.decoder`` runs a prompt and some steps of a
synthetic layer and prints the time of a step.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import PagedKVCache, kv_append, kv_attention, new_kv_workspace, rope_table, w4_matvec


@dataclass(frozen=True)
class LayerShape:
    model: int = 4096      # width of the residual stream
    q_heads: int = 32
    kv_heads: int = 8
    dim: int = 128         # of a head
    rot: int = 128         # elements of a head that are rotated
    group: int = 128       # codes that share a scale in the weights
    page: int = 64         # tokens of a cache page

    @property
    def fused(self) -> int:
        return (self.q_heads + 2 * self.kv_heads) * self.dim


def quantize4(w, group: int):
    """Codes, scales and zero points of float weights (n, k), for w4_matvec: each group's range
    in 15 steps, zero inside it."""
    n, k = w.shape
    groups = -(-k // group)
    padded = torch.zeros(n, groups * group, dtype=torch.float32, device=w.device)
    padded[:, :k] = w
    padded = padded.view(n, groups, group)
    lo, hi = padded.amin(-1).clamp(max=0.0), padded.amax(-1).clamp(min=0.0)
    scale = ((hi - lo) / 15.0).clamp(min=1e-8)
    zero = (-lo / scale).round().clamp(0, 15)
    codes = ((padded / scale[..., None]).round() + zero[..., None]).clamp(0, 15).to(torch.uint8).view(n, -1)[:, :k]
    if k % 2:
        codes = torch.nn.functional.pad(codes, (0, 1))
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous(), scale, zero.to(torch.uint8)


class AttentionLayer:
    """x + W_o attention(W_qkv x) over a batch of sequences that each own the pages of
    ``capacity`` tokens."""

    def __init__(self, shape: LayerShape, seqs: int, capacity: int, max_new: int, dtype=torch.bfloat16, codes=torch.int8,
                 seed: int = 0, device="cuda"):
        s = self.shape = shape
        self.seqs, self.dtype, self.max_new = seqs, dtype, max_new
        g = torch.Generator(device=device).manual_seed(seed)

        def weights(n, k):
            codes, scale, zero = quantize4(torch.randn(n, k, generator=g, device=device) * k ** -0.5, s.group)
            return codes, scale.to(dtype), zero

        self.qkv, self.out = weights(s.fused, s.model), weights(s.model, s.q_heads * s.dim)
        width = -(-capacity // s.page)
        self.cache = PagedKVCache.empty(seqs * width, s.kv_heads, s.page, s.dim, codes, device)
        # every sequence's pages are scattered over the cache, as an allocator would leave them
        self.block_table = torch.randperm(seqs * width, generator=g, device=device).to(torch.int32).view(seqs, width)
        self.ctx_len = torch.zeros(seqs, dtype=torch.int32, device=device)
        self.table = rope_table(capacity, s.rot, device=device)
        self.workspace = new_kv_workspace(self.cache, s.q_heads, max_new)
        self.one_each = torch.arange(seqs + 1, dtype=torch.int32, device=device)

    def run(self, x, counts=None, cu=None):
        """x (tokens, model), the new tokens of each sequence one after the other: counts (int32 [seqs]) of
        them with their offsets cu (int32 [seqs + 1]), or one each. Returns x's successor."""
        s = self.shape
        if cu is None:
            cu, most = self.one_each, 1
            self.ctx_len += 1
        else:
            most = self.max_new
            self.ctx_len += counts
        fused = w4_matvec(x, *self.qkv, group=s.group).view(-1, s.q_heads + 2 * s.kv_heads, s.dim)
        q, k, v = fused.split((s.q_heads, s.kv_heads, s.kv_heads), 1)
        q = kv_append(self.cache, q, k, v, self.table, self.block_table, self.ctx_len, cu, most, q_out=q)
        y = kv_attention(self.cache, q, self.block_table, self.ctx_len, cu, most, workspace=self.workspace)
        return w4_matvec(y.view(x.shape[0], -1), *self.out, group=s.group).add_(x)

    def capture(self, x):
        """A CUDA graph of one step on the buffer x (seqs, model), and the tensor that holds its
        result. One step runs before the capture, so that all kernels are loaded; no page is reached in it, whatever x holds:
        the cache and the lengths stay as they are."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        pages = self.block_table
        with torch.cuda.stream(side):
            self.block_table = torch.full_like(pages, -1)
            try:
                self.run(x)
                self.ctx_len -= 1
            finally:
                self.block_table = pages
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = self.run(x)
        return graph, y


def main():
    import time
    seqs, prompt, steps = 16, 500, 200
    layer = AttentionLayer(LayerShape(), seqs, prompt + 2 * steps, prompt)
    g = torch.Generator(device="cuda").manual_seed(1)
    counts = torch.full((seqs,), prompt, dtype=torch.int32, device="cuda")
    layer.run(torch.randn(seqs * prompt, layer.shape.model, generator=g, device="cuda").to(layer.dtype), counts,
              torch.arange(0, seqs * prompt + 1, prompt, dtype=torch.int32, device="cuda"))
    x = torch.randn(seqs, layer.shape.model, generator=g, device="cuda").to(layer.dtype)
    graph, _ = layer.capture(x)
    graph.replay()
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    print(f"{seqs} sequences of {prompt} tokens: {(time.perf_counter() - began) / steps * 1e6:.1f} us a step of one layer's attention")


if __name__ == "__main__":
    main()
