"""Decoding operators of a language model: products of a few rows with 4-bit
weights, the norms around a block with its gate and residual, and a paged 8-bit
cache of keys and values with its append (the position rotation applied on the way, on one
axis or several), attention (within a window, or to a prefix that sequences share) and read back.

Argument marshalling over include/om.h, like the rest of the binding: every
step of the computation is a kernel of the library. Tensors are CUDA tensors
with unit stride in the last dimension; activations are float32, float16 or
bfloat16; calls run on the current stream unless one is given (outputs that they
allocate then belong to that stream's memory, as under torch.cuda.stream), and never
synchronise. Sequences of a batch are given by ``cu`` (int32 [seqs + 1], sequence b has
tokens cu[b] .. cu[b + 1] - 1 of the call), ``ctx_len`` (int32 [seqs], its
length with those tokens) and ``block_table`` (int32 [seqs, width], the page of
each of its blocks).
"""
from __future__ import annotations

import ctypes

import torch

from . import OmError, lib

OM_F32, OM_F16, OM_BF16, OM_I8, OM_E4M3 = range(5)
DTYPES = {torch.float32: OM_F32, torch.float16: OM_F16, torch.bfloat16: OM_BF16}
CODES = {torch.int8: OM_I8, torch.float8_e4m3fn: OM_E4M3}
ROPE_SCALINGS = {None: 0, "plain": 0, "linear": 1, "ntk": 2, "yarn": 3}
NORMS = {"rms": 0, "layer": 1}
GATES = {None: 0, "none": 0, "sigmoid": 1, "silu": 2}
ROPE_PAIRS = {"half": 0, "interleaved": 1}


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("page", ctypes.c_int64), ("dim", ctypes.c_int64), ("dtype", ctypes.c_int)]


def _declare(L: ctypes.CDLL) -> None:
    i64, vp, ci, f32, f64 = (ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                             ctypes.c_double)
    L.om_w4_matvec.restype = ci
    L.om_w4_matvec.argtypes = [i64] * 4 + [vp, i64, ci, vp, i64, vp, i64, ci, vp, i64, vp, i64, vp]
    L.om_block_norm.restype = ci
    L.om_block_norm.argtypes = [i64, i64, vp, i64, ci, vp, i64, ci, vp, i64, ci, f32, ci, ci, f32, vp, vp, vp, vp, ci, vp, i64, vp, i64, vp]
    L.om_rope_table.restype = ci
    L.om_rope_table.argtypes = [i64, i64, f64, ci, f64, f64, f64, f64, vp, vp]
    L.om_kv_append.restype = ci
    append = [vp] + [i64] * 4 + [vp, i64, i64] * 3 + [ci, vp, i64, i64, ci, vp, i64, vp, vp, vp, i64, i64]
    L.om_kv_append.argtypes = append + [vp]
    L.om_kv_append_axes.restype = ci
    L.om_kv_append_axes.argtypes = append + [vp, i64, i64, vp, vp]
    L.om_kv_read.restype = ci
    L.om_kv_read.argtypes = [vp, i64, i64, vp, i64, vp, vp, vp, vp, ci, vp]
    L.om_kv_workspace_bytes.restype = ctypes.c_size_t
    L.om_kv_workspace_bytes.argtypes = [i64] * 4
    L.om_kv_attention.restype = ci
    batch, rest = [vp] + [i64] * 4 + [vp, i64, i64, ci, vp, i64, vp, vp, f32, i64], [vp, i64, i64, vp, vp, ctypes.c_size_t, vp]
    L.om_kv_attention.argtypes = batch + rest
    L.om_kv_attention_sinks.restype = ci
    L.om_kv_attention_sinks.argtypes = batch + [i64] + rest
    L.om_kv_shared_workspace_bytes.restype = ctypes.c_size_t
    L.om_kv_shared_workspace_bytes.argtypes = [i64] * 5
    L.om_kv_shared_attention.restype = ci
    L.om_kv_shared_attention.argtypes = [vp, i64, vp, i64, vp, vp] + [i64] * 4 + [vp, i64, i64, ci, vp, i64, vp, vp, f32] + rest


_functions = None


def _lib():
    """The loaded library (a name of this module once loaded: the calls here are short)."""
    global _functions
    if _functions is None:
        _functions = lib()
    return _functions


def _call(name, device, stream, *args):
    """Calls the library's function with the arguments and the stream (None: the device's current one) on a device,
    that of its tensors whichever is current, and raises on a status."""
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device) or None
    else:
        if stream.device_index != device:
            raise ValueError("stream and tensors are on different devices")
        handle = int(stream.cuda_stream) or None
    function = getattr(_lib(), name)
    if torch._C._cuda_getDevice() == device:
        st = function(*args, handle)
    else:
        with torch.cuda.device(device):
            st = function(*args, handle)
    if st:
        raise OmError(st, name)


def _empty(shape, dtype, device, stream):
    """A new output, of the memory that belongs to the stream that the call runs on: another stream's may still be read there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _like(t, stream):
    """A new output of a tensor's shape and type, contiguous."""
    if stream is None and t.is_contiguous():
        return torch.empty_like(t)
    return _empty(t.shape, t.dtype, t.device, stream)


def _cuda(t, name, dim, dtypes, device=None):
    """Raises unless t is a CUDA tensor of `dim` dimensions, one of the types and
    unit stride in the last dimension, on the device (by number) if one is given. Returns its device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a CUDA tensor of {' or '.join(str(d) for d in dtypes)}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} needs unit stride in its last dimension")
    on = t.get_device()
    if device is not None and on != device:
        raise ValueError(f"{name} is on another device")
    return on


_I32 = (torch.int32,)
_int32, _float32 = torch.int32, torch.float32


def w4_matvec(x, weight, scales, zeros=None, group: int = 128, out=None, stream=None):
    """x @ W.T for few rows of x and 4-bit W: W[j][p] = (code - zero) * scale.

    x (m, k); weight uint8 (n, (k + 1) // 2), the low half of a byte first; scales (n, ceil(k /
    group)) float32, float16 or bfloat16; zeros uint8 of that shape (None: 8
    everywhere); group 32, 64 or a multiple of 128. Returns (m, n) of x's type.
    """
    device = _cuda(x, "x", 2, DTYPES)
    _cuda(weight, "weight", 2, (torch.uint8,), device)
    _cuda(scales, "scales", 2, DTYPES, device)
    m, k = x.shape
    n, wb = weight.shape
    if group < 1:
        raise ValueError("group must be positive")
    groups = -(-k // group)
    if wb != (k + 1) // 2 or scales.shape != (n, groups):
        raise ValueError("weight, scales and x have different sizes")
    zp, ldz = None, 0
    if zeros is not None:
        _cuda(zeros, "zeros", 2, (torch.uint8,), device)
        if zeros.shape != (n, groups):
            raise ValueError("zeros and scales have different shapes")
        zp, ldz = zeros.data_ptr(), zeros.stride(0) if n > 1 else groups
    dtype = x.dtype
    if out is None:
        out = _empty((m, n), dtype, x.device, stream)
        ldy = n
    else:
        _cuda(out, "out", 2, (dtype,), device)
        if out.shape != (m, n):
            raise ValueError("out has the wrong shape")
        ldy = out.stride(0) if m > 1 else n
    if n > 1:
        wb, groups = weight.stride(0), scales.stride(0)
    _call("om_w4_matvec", device, stream, m, n, k, group, x.data_ptr(), x.stride(0) if m > 1 else k, DTYPES[dtype], weight.data_ptr(), wb,
          scales.data_ptr(), groups, DTYPES[scales.dtype], zp, ldz, out.data_ptr(), ldy)
    return out


def _vector(t, name, width, dtype, device):
    """Pointer of a (width,) operand."""
    if t.get_device() != device or t.dtype is not dtype or t.dim() != 1 or t.shape[0] != width or (width > 1 and t.stride(0) != 1):
        _cuda(t, name, 1, (dtype,), device)
        raise ValueError(f"{name} must have the shape ({width},)")
    return t.data_ptr()


def _rows(t, name, shape, dtype, device):
    """Pointer and row stride of a (tokens, width) operand."""
    if t.get_device() != device or t.dtype is not dtype or t.shape != shape:
        _cuda(t, name, 2, (dtype,), device)
        raise ValueError(f"{name} must have the shape {tuple(shape)}")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name} needs unit stride in its last dimension")
    return t.data_ptr(), ld if shape[0] > 1 else shape[1]


def block_norm(y, residual=None, weight=None, bias=None, *, post_weight=None, post_bias=None, gate=None, activation=None, scale: float = 1.0,
               norm: str = "rms", post=None, normed: bool = True, eps: float = 1e-6, sum_out=None, out=None, stream=None):
    """The norms before and after a block with its gate and residual scale: x = residual + scale *
    act(gate) * N_post(y) and h = N(x), in one pass. Returns (x, h).

    y (tokens, width), the block's output; residual of y's type or float32 (None: 0, and x is None unless sum_out is
    given: the norm before a first block is block_norm(x, weight=w)[1]); gate (tokens, width) or (width,) of y's type, activation
    None, "sigmoid" or "silu" of it; norm "rms" or "layer"; weights and biases (width,), all of y's type or all
    float32. post: whether y is normed (None: if it has a weight or bias); normed False: no second norm, h is None. sum_out (of the residual's type, y's
    without one) may be residual, out may be y. Widths of up to 32768.
    """
    device = _cuda(y, "y", 2, DTYPES)
    shape, dtype = y.shape, y.dtype
    width = shape[1]
    if norm not in NORMS:
        raise ValueError(f"unknown norm {norm!r}")
    if activation not in GATES:
        raise ValueError(f"unknown activation {activation!r}")
    stream_dtype = dtype
    rp, ldr = None, 0
    if residual is not None:
        if residual.dtype is _float32:
            stream_dtype = _float32
        rp, ldr = _rows(residual, "residual", shape, stream_dtype, device)
    elif sum_out is not None and sum_out.dtype is _float32:
        stream_dtype = _float32
    gp, ldg = None, 0
    if gate is None:
        if GATES[activation]:
            raise ValueError("an activation needs a gate")
    elif gate.dim() == 1:
        gp = _vector(gate, "gate", width, dtype, device)
    else:
        gp, ldg = _rows(gate, "gate", shape, dtype, device)
    weight_dtype = dtype
    for w in (weight, post_weight, bias, post_bias):
        if w is not None:
            if w.dtype is _float32:
                weight_dtype = _float32
            break
    wp = None if weight is None else _vector(weight, "weight", width, weight_dtype, device)
    bp = None if bias is None else _vector(bias, "bias", width, weight_dtype, device)
    pwp = None if post_weight is None else _vector(post_weight, "post_weight", width, weight_dtype, device)
    pbp = None if post_bias is None else _vector(post_bias, "post_bias", width, weight_dtype, device)
    if post is None:
        post = post_weight is not None or post_bias is not None
    sp, lds, op, ldo = None, 0, None, 0
    if residual is not None or sum_out is not None:
        if sum_out is None:
            sum_out = _like(residual, stream)
            sp, lds = sum_out.data_ptr(), width
        else:
            sp, lds = _rows(sum_out, "sum_out", shape, stream_dtype, device)
    elif not normed:
        raise ValueError("nothing to compute: no residual, no sum_out and no second norm")
    if normed:
        if out is None:
            out = _like(y, stream)
            op, ldo = out.data_ptr(), width
        else:
            op, ldo = _rows(out, "out", shape, dtype, device)
    elif weight is not None or bias is not None or out is not None:
        raise ValueError("weight, bias and out belong to the second norm")
    _call("om_block_norm", device, stream, shape[0], width, y.data_ptr(), y.stride(0) if shape[0] > 1 else width, DTYPES[dtype], rp, ldr,
          DTYPES[stream_dtype], gp, ldg, GATES[activation], scale, NORMS[norm], post, eps, pwp, pbp, wp, bp, DTYPES[weight_dtype], sp, lds, op, ldo)
    return sum_out, out


def rope_table(rows: int, rot: int, base: float = 10000.0, scaling=None, factor: float = 1.0,
               original: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda",
               stream=None):
    """cos and sin of each position's angles, float32 (rows, rot // 2, 2), evaluated in 64
    bits. scaling: None, "linear", "ntk" or "yarn" (see om_rope_table)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"unknown scaling {scaling!r}")
    out = _empty((rows, rot // 2, 2), torch.float32, device, stream)
    _call("om_rope_table", _cuda(out, "device's memory", 3, (torch.float32,)), stream, rows, rot, base, ROPE_SCALINGS[scaling], factor, original,
          beta_fast, beta_slow, out.data_ptr())
    return out


class PagedKVCache:
    """Keys and values in 8 bits: codes (pages, heads, page, dim) of int8 or
    float8_e4m3fn and one float32 scale per page and head, (pages, heads). A
    handle: it owns references to the four tensors, which stay the caller's."""

    def __init__(self, k, v, k_scale, v_scale):
        for t, name, dim, dtypes in ((k, "k", 4, CODES), (v, "v", 4, CODES), (k_scale, "k_scale", 2, (torch.float32,)),
                                     (v_scale, "v_scale", 2, (torch.float32,))):
            self.device = _cuda(t, name, dim, dtypes, k.get_device())
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if k.shape != v.shape or k.dtype != v.dtype or k_scale.shape != k.shape[:2] or v_scale.shape != k.shape[:2]:
            raise ValueError("keys, values and scales have different shapes or types")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.page, self.dim = k.shape
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), *k.shape,
                                    CODES[k.dtype])
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, pages: int, heads: int, page: int, dim: int, dtype=torch.int8, device="cuda"):
        """A cache that holds nothing yet."""
        k, v = (torch.zeros((pages, heads, page, dim), dtype=torch.int8, device=device).view(dtype) for _ in range(2))
        ks, vs = (torch.zeros((pages, heads), dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)


def _batch(block_table, lens, cu, lens_name, device, table_name="block_table", cu_name="cu"):
    """Pointers and sizes of a batch's lookups: (block_table, width, lens, cu), sequences."""
    if not (block_table.get_device() == lens.get_device() == cu.get_device() == device and block_table.dtype is lens.dtype is cu.dtype is _int32
            and block_table.dim() == 2 and lens.dim() == 1 and cu.dim() == 1 and block_table.is_contiguous() and lens.is_contiguous()
            and cu.is_contiguous()):
        _cuda(block_table, table_name, 2, _I32, device)
        _cuda(lens, lens_name, 1, _I32, device)
        _cuda(cu, cu_name, 1, _I32, device)
        raise ValueError(f"{table_name} must be contiguous")
    seqs, width = block_table.shape
    if lens.numel() != seqs or cu.numel() != seqs + 1:
        raise ValueError(f"{table_name}, {lens_name} and {cu_name} are of different batches")
    return (block_table.data_ptr(), width, lens.data_ptr(), cu.data_ptr()), seqs


def _heads(t, name, shape, dtype, device):
    """Pointer, token stride and head stride of a (tokens, heads, dim) operand."""
    if t.get_device() != device or t.dtype is not dtype or t.shape != shape:
        _cuda(t, name, 3, (dtype,), device)
        raise ValueError(f"{name} must have the shape {tuple(shape)}")
    ts, hs, one = t.stride()
    if one != 1:
        raise ValueError(f"{name} needs unit stride in its last dimension")
    return t.data_ptr(), ts, hs


def rope_axes(sections, order: str = "blocks", device="cuda"):
    """The axis that turns each rotated pair, int32 (sum of sections,), for kv_append: sections[a] pairs of axis
    a, one axis after the other ("blocks"), or in turns as long as each has pairs left ("turns")."""
    sections = [int(n) for n in sections]
    if order not in ("blocks", "turns"):
        raise ValueError(f"unknown order {order!r}")
    if not sections or min(sections) < 0:
        raise ValueError("sections must be numbers of pairs")
    if order == "blocks":
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    else:
        axis = [a for i in range(max(sections)) for a, n in enumerate(sections) if i < n]
    return torch.tensor(axis, dtype=torch.int32, device=device)


def kv_append(cache, q, k, v, table, block_table, ctx_len, cu, max_new: int, pairs: str = "half", q_out=None,
              stream=None, positions=None, pair_axis=None):
    """Stores the new tokens' keys (rotated) and values in the cache and returns the
    rotated queries.

    q (tokens, q heads, dim) or None, k and v (tokens, heads, dim) may be parts of one buffer; table
    from rope_table (None: no rotation); max_new at least the largest number of new
    tokens of a sequence. q_out may be q.

    positions, int32 (axes, tokens): the tokens' rotary positions on each axis, where these are not their places in the
    cache (patches of images and videos; None: the places). pair_axis, int32 (rot // 2,): the axis
    that turns each pair, as rope_axes lays them out (None: axis 0).
    """
    device = cache.device
    _cuda(k, "k", 3, DTYPES, device)
    dtype, tokens, dim = k.dtype, k.shape[0], cache.dim
    shape = (tokens, cache.heads, dim)
    ka, va = _heads(k, "k", shape, dtype, device), _heads(v, "v", shape, dtype, device)
    batch, seqs = _batch(block_table, ctx_len, cu, "ctx_len", device)
    if pairs not in ROPE_PAIRS:
        raise ValueError(f"unknown pairs {pairs!r}")
    qa, oa, q_heads = (None, 0, 0), (None, 0, 0), 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must have 3 dimensions")
        q_heads = q.shape[1]
        shape = (tokens, q_heads, dim)
        qa = _heads(q, "q", shape, dtype, device)
        if q_out is None:
            q_out = _empty(shape, dtype, q.device, stream)
            oa = q_out.data_ptr(), q_heads * dim, dim
        else:
            oa = _heads(q_out, "q_out", shape, dtype, device)
    tp, rows, rot = None, 0, 0
    if table is not None:
        _cuda(table, "table", 3, (torch.float32,), device)
        rows, rot, two = table.shape
        if two != 2 or not table.is_contiguous():
            raise ValueError("table must be a contiguous (rows, rot // 2, 2) tensor")
        tp, rot = table.data_ptr(), 2 * rot
    args = cache._ref, seqs, tokens, max_new, q_heads, *qa, *ka, *va, DTYPES[dtype], tp, rows, rot, ROPE_PAIRS[pairs], *batch, *oa
    if positions is None:
        if pair_axis is not None:
            raise ValueError("pair_axis needs positions")
        _call("om_kv_append", device, stream, *args)
        return q_out
    _cuda(positions, "positions", 2, _I32, device)
    axes = positions.shape[0]
    if positions.shape[1] != tokens or axes < 1:
        raise ValueError("positions must have the shape (axes, tokens)")
    ap = None
    if pair_axis is not None:
        _cuda(pair_axis, "pair_axis", 1, _I32, device)
        if pair_axis.shape[0] * 2 != rot:
            raise ValueError("pair_axis must have an axis for each pair of the table")
        ap = pair_axis.data_ptr()
    _call("om_kv_append_axes", device, stream, *args, positions.data_ptr(), axes, positions.stride(0) if axes > 1 else tokens, ap)
    return q_out


def kv_read(cache, block_table, start, cu, max_tokens: int, tokens: int, dtype=torch.float32, k_out=None, v_out=None,
            stream=None):
    """Reads `tokens` tokens back as values: token i of sequence b is position
    start[b] + i. The lengths come from cu; max_tokens, at least the largest of them, is not
    needed for them. Returns keys and values, (tokens, heads, dim) of dtype."""
    device = cache.device
    batch, seqs = _batch(block_table, start, cu, "start", device)
    if dtype not in DTYPES:
        raise TypeError("dtype must be float32, float16 or bfloat16")
    if tokens < 0 or max_tokens < 0:
        raise ValueError("tokens and max_tokens must not be negative")
    shape = (tokens, cache.heads, cache.dim)
    if k_out is None:
        k_out = _empty(shape, dtype, block_table.device, stream)
    else:
        _heads(k_out, "k_out", shape, dtype, device)
    if v_out is None:
        v_out = _empty(shape, dtype, block_table.device, stream)
    else:
        _heads(v_out, "v_out", shape, dtype, device)
    if not (k_out.is_contiguous() and v_out.is_contiguous()):
        raise ValueError("k_out and v_out must be contiguous")
    _call("om_kv_read", device, stream, cache._ref, seqs, tokens, *batch, k_out.data_ptr(), v_out.data_ptr(), DTYPES[dtype])
    return k_out, v_out


def new_kv_workspace(cache, q_heads: int, max_new: int):
    """A device tensor usable as the workspace of kv_attention for calls of these
    heads with at most max_new queries a sequence; one per stream."""
    n = lib().om_kv_workspace_bytes(cache.heads, q_heads, cache.dim, max_new)
    if n == 0:
        raise ValueError("q_heads must be a multiple of the cache's heads, max_new positive")
    return torch.zeros((n + 3) // 4, dtype=torch.int32, device=cache.k.device)


def kv_attention(cache, q, block_table, ctx_len, cu, max_new: int, scale=None, window: int = 0, out=None, lse=None,
                 workspace=None, stream=None, sinks: int = 0):
    """Attention of each sequence's last tokens' queries, q (tokens, q heads, dim),
    to its cached tokens, causal, within `window` positions (0: all) and the sequence's first `sinks` ones (a mask: they keep the
    rotation that they were stored with).

    scale: default dim ** -0.5. lse: float32 (tokens, q heads), receives the natural log of the sums
    of exponentials. workspace: from new_kv_workspace; without one each sequence
    and head is one block's work. Rows of tokens behind cu's last offset are not written. Returns (tokens, q heads,
    dim) of q's type.
    """
    device = cache.device
    _cuda(q, "q", 3, DTYPES, device)
    dtype, shape = q.dtype, q.shape
    tokens, q_heads, dim = shape
    if dim != cache.dim:
        raise ValueError("q and the cache have different head dimensions")
    ts, hs, _ = q.stride()
    batch, seqs = _batch(block_table, ctx_len, cu, "ctx_len", device)
    if out is None:
        out = _empty(shape, dtype, q.device, stream)
        oa = out.data_ptr(), q_heads * dim, dim
    else:
        oa = _heads(out, "out", shape, dtype, device)
    lp = None
    if lse is not None:
        _cuda(lse, "lse", 2, (torch.float32,), device)
        if lse.shape != (tokens, q_heads) or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous (tokens, q heads) tensor")
        lp = lse.data_ptr()
    ws, ws_bytes = None, 0
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the cache's device")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    name, visible = ("om_kv_attention_sinks", (window, sinks)) if sinks else ("om_kv_attention", (window,))
    _call(name, device, stream, cache._ref, seqs, tokens, max_new, q_heads, q.data_ptr(), ts, hs, DTYPES[dtype], *batch,
          dim ** -0.5 if scale is None else scale, *visible, *oa, lp, ws, ws_bytes)
    return out


def new_shared_workspace(cache, q_heads: int, max_new: int, tokens: int):
    """A device tensor usable as the workspace of kv_shared_attention for calls of these heads
    with at most `tokens` tokens and max_new queries a sequence; one per stream. It holds 8 dim + 16 bytes for each token and
    query head: 2.2 GB for 65536 tokens of 32 heads of 128."""
    n = lib().om_kv_shared_workspace_bytes(cache.heads, q_heads, cache.dim, max_new, tokens)
    if n == 0:
        raise ValueError("q_heads must be a multiple of the cache's heads, max_new and tokens positive")
    return torch.zeros((n + 3) // 4, dtype=torch.int32, device=cache.k.device)


def kv_shared_attention(cache, q, prefix_table, prefix_len, groups, block_table, ctx_len, cu, max_new: int, scale=None, out=None, lse=None,
                        workspace=None, stream=None):
    """kv_attention of a batch whose sequences share prefixes, each of which is read once for all of them.

    groups (int32 [prefixes + 1], not decreasing): sequences groups[j] .. groups[j + 1] - 1 begin with the prefix_len[j] tokens
    (int32 [prefixes]) in the pages prefix_table[j] (int32 [prefixes, width]); block_table, ctx_len and cu are
    the sequences' own tokens behind it, which start on a page of their own. A query sees its whole
    prefix and its sequence's own tokens up to itself. workspace: from new_shared_workspace (None: a new one, zeroed as a whole in
    every call). A prefix_table that is no wider than its prefixes need does best. scale, lse,
    and what is returned, as in kv_attention.
    """
    device = cache.device
    _cuda(q, "q", 3, DTYPES, device)
    dtype, shape = q.dtype, q.shape
    tokens, q_heads, dim = shape
    if dim != cache.dim:
        raise ValueError("q and the cache have different head dimensions")
    ts, hs, _ = q.stride()
    batch, seqs = _batch(block_table, ctx_len, cu, "ctx_len", device)
    (pp, pwidth, lens, offsets), count = _batch(prefix_table, prefix_len, groups, "prefix_len", device, "prefix_table", "groups")
    if out is None:
        out = _empty(shape, dtype, q.device, stream)
        oa = out.data_ptr(), q_heads * dim, dim
    else:
        oa = _heads(out, "out", shape, dtype, device)
    lp = None
    if lse is not None:
        _cuda(lse, "lse", 2, (torch.float32,), device)
        if lse.shape != (tokens, q_heads) or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous (tokens, q heads) tensor")
        lp = lse.data_ptr()
    if tokens == 0 or seqs == 0:
        return out
    if workspace is None:
        n = _lib().om_kv_shared_workspace_bytes(cache.heads, q_heads, dim, max_new, tokens)
        with torch.cuda.stream(stream):
            workspace = torch.zeros((n + 3) // 4, dtype=torch.int32, device=q.device)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    _call("om_kv_shared_attention", device, stream, cache._ref, count, pp, pwidth, lens, offsets, seqs, tokens, max_new, q_heads, q.data_ptr(), ts, hs,
          DTYPES[dtype], *batch, dim ** -0.5 if scale is None else scale, *oa, lp, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out
