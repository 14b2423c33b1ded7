"""The attention half of a decoder layer on the decoding operators: 4-bit products,
the append to a paged 8-bit cache with the position rotation, and attention over it.

One call of :meth:`AttentionLayer.run` takes any number of new tokens of each sequence: a
prompt, or one token of every sequence (:meth:`AttentionLayer.capture` makes a CUDA
graph of that step; lengths live on the device and grow with every replay). The
operators are the library's; what is torch here is bookkeeping (slicing the fused
projection, adding the residual of a layer without norms, counting positions).

A layer can have norms before and after its attention (with a gate for each channel and a residual scale),
a sliding window whose first tokens stay visible, rotary positions of several axes (images and videos), and a
prefix that all its sequences share (:meth:`AttentionLayer.run_prefix`, once; it is kept once and attended once a step).

``python -m implicit_gemm_convolution_gb300.decoder`` runs a prompt and some steps of a
synthetic layer and prints the time of a step.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (PagedKVCache, block_norm, kv_append, kv_attention, kv_shared_attention, new_kv_workspace, new_shared_workspace, rope_axes, rope_table,
               w4_matvec)


@dataclass(frozen=True)
class LayerShape:
    model: int = 4096      # width of the residual stream
    q_heads: int = 32
    kv_heads: int = 8
    dim: int = 128         # of a head
    rot: int = 128         # elements of a head that are rotated
    group: int = 128       # codes that share a scale in the weights
    page: int = 64         # tokens of a cache page
    norm: str | None = None  # "rms" or "layer": a norm before the attention
    post_norm: bool = False  # and one after it, before the residual
    gate: bool = False       # a factor for each channel of the block's output
    residual_scale: float = 1.0
    window: int = 0        # positions that a token sees, itself among them (0: all)
    sinks: int = 0         # a sequence's first tokens, which a window leaves visible
    sections: tuple = ()   # rotated pairs of each axis of positions (): one axis, the token's place
    order: str = "blocks"  # of the axes, as in rope_axes

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


def places(ctx_len, cu, tokens: int):
    """The place of each of a call's tokens in its sequence, int32 (tokens,), found on the device: the sequence's new tokens are its
    last ones. Rows behind the last sequence's tokens, which a padded batch has, count on from it."""
    token = torch.arange(tokens, dtype=torch.int32, device=cu.device)
    seq = torch.searchsorted(cu[1:], token, right=True).clamp_(max=max(ctx_len.shape[0] - 1, 0))
    return token + (ctx_len - cu[1:])[seq]


class AttentionLayer:
    """x + W_o attention(W_qkv x), or x + scale gate N_post(W_o attention(W_qkv N(x))) with norms, over a batch of sequences
    that each own the pages of ``capacity`` tokens, behind a common prefix of up to ``prefix`` tokens."""

    def __init__(self, shape: LayerShape, seqs: int, capacity: int, max_new: int, dtype=torch.bfloat16, codes=torch.int8,
                 seed: int = 0, device="cuda", prefix: int = 0):
        s = self.shape = shape
        if prefix and s.window:
            raise ValueError("a window and a shared prefix do not go together")
        if not s.norm and (s.post_norm or s.gate or s.residual_scale != 1.0):
            raise ValueError("post_norm, gate and residual_scale belong to a layer with norms")
        if s.sections and 2 * sum(s.sections) != s.rot:
            raise ValueError("sections must have an axis for each rotated pair")
        self.seqs, self.dtype, self.max_new, self.prefix = seqs, dtype, max_new, prefix
        g = torch.Generator(device=device).manual_seed(seed)

        def weights(n, k):
            codes, scale, zero = quantize4(torch.randn(n, k, generator=g, device=device) * k ** -0.5, s.group)
            return codes, scale.to(dtype), zero

        self.qkv, self.out = weights(s.fused, s.model), weights(s.model, s.q_heads * s.dim)
        width, shared = -(-capacity // s.page), -(-prefix // s.page)
        self.cache = PagedKVCache.empty(seqs * width + shared, s.kv_heads, s.page, s.dim, codes, device)
        # every sequence's pages are scattered over the cache, as an allocator would leave them
        pages = torch.randperm(seqs * width + shared, generator=g, device=device).to(torch.int32)
        self.block_table, self.prefix_table = pages[: seqs * width].view(seqs, width), pages[seqs * width:].view(1, shared)
        self.ctx_len = torch.zeros(seqs, dtype=torch.int32, device=device)
        self.table = rope_table(capacity + prefix, s.rot, device=device)
        self.one_each = torch.arange(seqs + 1, dtype=torch.int32, device=device)
        self.prefix_len, self.groups = (torch.tensor(v, dtype=torch.int32, device=device) for v in ([0], [0, seqs]))
        if prefix:
            self.workspace = new_shared_workspace(self.cache, s.q_heads, max_new, seqs * max_new)
        else:
            self.workspace = new_kv_workspace(self.cache, s.q_heads, max_new)
        self.axis = rope_axes(s.sections, s.order, device) if s.sections else None

        def vector(there, around):
            return (around + 0.1 * torch.randn(s.model, generator=g, device=device)).to(dtype) if there else None

        self.norm_weight, self.post_weight, self.gate = vector(s.norm, 1.0), vector(s.post_norm, 1.0), vector(s.gate, 1.0)

    def run(self, x, counts=None, cu=None, positions=None):
        """x (tokens, model), the new tokens of each sequence one after the other: counts (int32 [seqs]) of
        them with their offsets cu (int32 [seqs + 1]; rows of x behind them are nobody's, and what comes back there is not
        defined), or one each. positions (int32 [axes, tokens]): the tokens' rotary
        positions on each axis, for a layer with sections (None: their places, on all axes). Returns x's successor."""
        step = cu is None
        if step:
            cu, most = self.one_each, 1
            self.ctx_len += 1
        else:
            most = self.max_new
            self.ctx_len += counts
        if positions is None and (self.axis is not None or self.prefix_table.shape[1]):
            # places in the sequence, the prefix among them
            own = self.ctx_len - 1 if step else places(self.ctx_len, cu, x.shape[0])
            positions = (own + self.prefix_len).expand(len(self.shape.sections) or 1, -1).contiguous()
        return self._block(x, self.block_table, self.ctx_len, cu, most, positions, self.prefix_table.shape[1] > 0)

    def run_prefix(self, x, positions=None):
        """The prefix that all sequences share, x (tokens, model): computed and kept once, before the sequences' own
        tokens. Returns x's successor."""
        tokens = x.shape[0]
        # the last page may have room for more, but the rotation's table has none for the own tokens behind them
        if not 0 < tokens <= self.prefix:
            raise ValueError("the layer has no room for such a prefix")
        if positions is None and self.axis is not None:
            positions = torch.arange(tokens, dtype=torch.int32, device=x.device).expand(len(self.shape.sections), -1).contiguous()
        self.prefix_len.fill_(tokens)
        cu = torch.tensor([0, tokens], dtype=torch.int32, device=x.device)
        return self._block(x, self.prefix_table, self.prefix_len, cu, tokens, positions, False)

    def _block(self, x, block_table, ctx_len, cu, most, positions, shared):
        s = self.shape
        h = block_norm(x, weight=self.norm_weight, norm=s.norm)[1] if s.norm else x
        fused = w4_matvec(h, *self.qkv, group=s.group).view(-1, s.q_heads + 2 * s.kv_heads, s.dim)
        q, k, v = fused.split((s.q_heads, s.kv_heads, s.kv_heads), 1)
        q = kv_append(self.cache, q, k, v, self.table, block_table, ctx_len, cu, most, q_out=q, positions=positions,
                      pair_axis=self.axis if positions is not None else None)
        if shared:
            y = kv_shared_attention(self.cache, q, self.prefix_table, self.prefix_len, self.groups, block_table, ctx_len, cu, most, workspace=self.workspace)
        else:
            # a prefix's own queries are more than the workspace was made for: each item by one block
            y = kv_attention(self.cache, q, block_table, ctx_len, cu, most, workspace=self.workspace if block_table is self.block_table else None,
                             window=s.window, sinks=s.sinks)
        y = w4_matvec(y.view(x.shape[0], -1), *self.out, group=s.group)
        if not s.norm:
            return y.add_(x)
        return block_norm(y, x, post_weight=self.post_weight, gate=self.gate, scale=s.residual_scale, norm=s.norm, normed=False)[0]

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
