// decode_api.cu -- the C ABI of the decoding operators: argument validation and launch
// on the caller's stream. Nothing is launched by a call that fails validation.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "decode.h"
#include "om.h"
#include "om_internal.h"

namespace {

using om::Heads;

constexpr int64_t kLim31 = (int64_t(1) << 31) - 1;
constexpr int64_t kMargin = int64_t(1) << 16;  // positions and rows are rounded up in 32 bits

int from_cuda(cudaError_t e) { return e == cudaSuccess ? OM_OK : OM_ERR_CUDA; }

bool float_type(int t) { return t == OM_F32 || t == OM_F16 || t == OM_BF16; }
int64_t type_bytes(int t) { return t == OM_F32 ? 4 : (t == OM_F16 || t == OM_BF16 ? 2 : 1); }
bool aligned(const void *p, int64_t to) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(to) == 0; }

// The bytes of a block of `rows` rows of `row` bytes, `stride` bytes apart.
struct Block {
    uintptr_t lo = 0;
    int64_t rows = 0, row = 0, stride = 0;
    uintptr_t hi() const { return rows <= 0 || row <= 0 ? lo : lo + static_cast<uintptr_t>((rows - 1) * stride + row); }
};

// Whether two blocks share a byte. Blocks of one row stride whose rows fit
// beside each other in it (the parts of a fused buffer) do not.
bool overlaps(const Block &a, const Block &b) {
    if (a.lo == a.hi() || b.lo == b.hi() || a.lo >= b.hi() || b.lo >= a.hi()) return false;
    if (a.rows > 1 && b.rows > 1 && a.stride == b.stride && a.row <= a.stride && b.row <= b.stride) {
        const int64_t d = static_cast<int64_t>((b.lo >= a.lo ? b.lo - a.lo : a.lo - b.lo) % static_cast<uintptr_t>(a.stride));
        const int64_t from = b.lo >= a.lo ? d : (a.stride - d) % a.stride;  // b's rows start this far into a's
        return from < a.row || from + b.row > a.stride;
    }
    return true;
}

Block flat(const void *p, __int128 bytes) {
    Block b;
    b.lo = reinterpret_cast<uintptr_t>(p);
    b.rows = bytes > 0 ? 1 : 0;
    b.row = b.stride = static_cast<int64_t>(bytes);
    return b;
}

Block rows_of(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t bytes) {
    Block b;
    b.lo = reinterpret_cast<uintptr_t>(p);
    b.rows = cols > 0 ? rows : 0;
    b.row = cols * bytes;
    b.stride = rows > 1 ? ld * bytes : b.row;  // the stride of a single row may be anything
    return b;
}

// A [tokens][heads][dim] operand: strides that are not negative, extents below 2^60.
int check_heads(const Heads &x, int64_t tokens, int64_t heads, int64_t dim, int dtype, bool out) {
    if (!x.p) return OM_ERR_NULL_PTR;
    if (x.ts < 0 || x.hs < 0) return OM_ERR_INVALID_ARG;
    if ((heads > 1 && x.hs < dim) || (out && tokens > 1 && x.ts < (heads - 1) * x.hs + dim)) return OM_ERR_INVALID_ARG;
    const __int128 e = static_cast<__int128>(tokens - 1) * x.ts + static_cast<__int128>(heads - 1) * x.hs + dim;
    if (e >= (static_cast<__int128>(1) << 60)) return OM_ERR_TOO_LARGE;
    return aligned(x.p, type_bytes(dtype)) ? OM_OK : OM_ERR_ALIGNMENT;
}

Block heads_block(const Heads &x, int64_t tokens, int64_t heads, int64_t dim, int dtype) {
    return rows_of(x.p, tokens, (heads - 1) * (heads > 1 ? x.hs : 0) + dim, x.ts, type_bytes(dtype));
}

int check_cache(const om_kv_cache *c) {
    if (!c) return OM_ERR_NULL_PTR;
    if (c->pages < 0 || c->heads < 1) return OM_ERR_INVALID_ARG;
    if (c->dtype != OM_I8 && c->dtype != OM_E4M3) return OM_ERR_UNSUPPORTED;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return OM_ERR_UNSUPPORTED;
    if (c->dim != 64 && c->dim != 128 && c->dim != 256) return OM_ERR_UNSUPPORTED;
    if (c->pages > kLim31 || c->heads > 65535) return OM_ERR_TOO_LARGE;
    if (c->pages > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return OM_ERR_NULL_PTR;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return OM_ERR_ALIGNMENT;
    return OM_OK;
}

struct CacheBlocks {
    Block b[4];
    explicit CacheBlocks(const om_kv_cache &c) {
        const __int128 codes = static_cast<__int128>(c.pages) * c.heads * c.page * c.dim;
        const __int128 scales = static_cast<__int128>(c.pages) * c.heads * 4;
        b[0] = flat(c.k, codes); b[1] = flat(c.v, codes); b[2] = flat(c.k_scale, scales); b[3] = flat(c.v_scale, scales);
    }
    bool overlap(const Block &x) const {
        for (const Block &y : b)
            if (overlaps(x, y)) return true;
        return false;
    }
    bool overlap_themselves() const {
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < i; ++j)
                if (overlaps(b[i], b[j])) return true;
        return false;
    }
};

// The batch's lookups: block table, lengths and token offsets.
int check_batch(int64_t seqs, int64_t tokens, const int32_t *block_table, int64_t width, int64_t page,
                const int32_t *lens, const int32_t *cu) {
    if (!block_table || !lens || !cu) return OM_ERR_NULL_PTR;
    if (width < 1) return OM_ERR_INVALID_ARG;
    if (seqs > kLim31 || tokens > kLim31 || width > (kLim31 - kMargin) / page) return OM_ERR_TOO_LARGE;
    return aligned(block_table, 4) && aligned(lens, 4) && aligned(cu, 4) ? OM_OK : OM_ERR_ALIGNMENT;
}

struct BatchBlocks {
    Block b[3];
    BatchBlocks(int64_t seqs, const int32_t *table, int64_t width, const int32_t *lens, const int32_t *cu) {
        b[0] = flat(table, static_cast<__int128>(seqs) * width * 4);
        b[1] = flat(lens, static_cast<__int128>(seqs) * 4);
        b[2] = flat(cu, static_cast<__int128>(seqs + 1) * 4);
    }
    bool overlap(const Block &x) const { return overlaps(x, b[0]) || overlaps(x, b[1]) || overlaps(x, b[2]); }
};

// Where a call on shared prefixes keeps what its kernels hand on, behind the scratch of the attention to own tokens.
struct SharedPlaces {
    float2 *whole_state, *own_state, *slot_state;
    float *whole, *own, *slots, *kept;
    int64_t slot_rows;
    size_t bytes;
};
SharedPlaces shared_places(void *workspace, int64_t group, int64_t q_heads, int64_t dim, int64_t max_new, int64_t tokens) {
    size_t used = om::kv_workspace_bytes(group, dim, max_new);
    auto take = [&](int64_t bytes) {
        used = (used + 15) / 16 * 16;
        uint8_t *const at = static_cast<uint8_t *>(workspace) + used;
        used += static_cast<size_t>(bytes);
        return workspace ? at : nullptr;
    };
    SharedPlaces p{};
    const int64_t rows = tokens * q_heads;
    p.slot_rows = tokens * group < om::kSharedRows ? tokens * group : om::kSharedRows;
    const int64_t slots = 2 * om::kSharedMostBlocks * p.slot_rows;
    p.whole_state = reinterpret_cast<float2 *>(take(rows * 8));
    p.own_state = reinterpret_cast<float2 *>(take(rows * 8));
    p.slot_state = reinterpret_cast<float2 *>(take(slots * 8));
    p.whole = reinterpret_cast<float *>(take(rows * dim * 4));
    p.own = reinterpret_cast<float *>(take(rows * dim * 4));
    p.slots = reinterpret_cast<float *>(take(slots * dim * 4));
    p.kept = reinterpret_cast<float *>(take(slots / 2 * dim * 4));
    p.bytes = used;
    return p;
}

bool same(const Heads &a, const Heads &b) { return a.p == b.p && a.ts == b.ts && a.hs == b.hs; }

}  // namespace

extern "C" {

int om_w4_matvec(int64_t m, int64_t n, int64_t k, int64_t group, const void *x, int64_t ldx, int x_dtype,
                 const uint8_t *w, int64_t ldw, const void *scales, int64_t lds, int scale_dtype,
                 const uint8_t *zeros, int64_t ldz, void *y, int64_t ldy, void *stream) {
    if (m < 0 || n < 0 || k < 0 || group < 1) return OM_ERR_INVALID_ARG;
    if (!float_type(x_dtype) || !float_type(scale_dtype)) return OM_ERR_UNSUPPORTED;
    if (group != 32 && group != 64 && group % 128 != 0) return OM_ERR_UNSUPPORTED;
    if (m == 0 || n == 0) return OM_OK;
    // 16 rows of weights and scales are below 2^31 bytes
    const int64_t row_lim = int64_t(1) << 26;
    if (m > 65535 || n > kLim31 - 256 || k > row_lim || group > kLim31) return OM_ERR_TOO_LARGE;
    const int64_t groups = (k + group - 1) / group, wb = (k + 1) / 2;
    if (ldy < n || (k > 0 && (ldx < k || ldw < wb || lds < groups || (zeros && ldz < groups)))) return OM_ERR_INVALID_ARG;
    if (!y || (k > 0 && (!x || !w || !scales))) return OM_ERR_NULL_PTR;
    const int64_t big = int64_t(1) << 40;
    if (ldy > big || ldx > big || ldw > row_lim || lds > row_lim / 4 || (zeros && ldz > row_lim)) return OM_ERR_TOO_LARGE;
    const int64_t xb = type_bytes(x_dtype), sb = type_bytes(scale_dtype);
    if (!aligned(y, xb) || !aligned(x, xb) || !aligned(scales, sb)) return OM_ERR_ALIGNMENT;
    const Block ry = rows_of(y, m, n, ldy, xb);
    if (k > 0 && (overlaps(ry, rows_of(x, m, k, ldx, xb)) || overlaps(ry, rows_of(w, n, wb, ldw, 1)) ||
                  overlaps(ry, rows_of(scales, n, groups, lds, sb)) ||
                  (zeros && overlaps(ry, rows_of(zeros, n, groups, ldz, 1)))))
        return OM_ERR_ALIAS;
    const om::W4Problem p{m, n, k, group, x, ldx, x_dtype, w, ldw, scales, lds, scale_dtype, zeros, ldz, y, ldy};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (x_dtype == OM_F32) return from_cuda(om::launch_w4_matvec_f32(p, st));
    return from_cuda(x_dtype == OM_F16 ? om::launch_w4_matvec_f16(p, st) : om::launch_w4_matvec_bf16(p, st));
}

int om_block_norm(int64_t tokens, int64_t width, const void *y, int64_t ldy, int dtype, const void *residual, int64_t ldr, int stream_dtype,
                  const void *gate, int64_t ldg, int activation, float scale, int norm, int post, float eps, const void *post_weight,
                  const void *post_bias, const void *weight, const void *bias, int weight_dtype, void *sum, int64_t lds, void *out, int64_t ldo,
                  void *stream) {
    if (tokens < 0 || width < 0) return OM_ERR_INVALID_ARG;
    if (!float_type(dtype) || !float_type(stream_dtype) || !float_type(weight_dtype)) return OM_ERR_UNSUPPORTED;
    if ((stream_dtype != dtype && stream_dtype != OM_F32) || (weight_dtype != dtype && weight_dtype != OM_F32)) return OM_ERR_UNSUPPORTED;
    if (norm != OM_NORM_RMS && norm != OM_NORM_LAYER) return OM_ERR_UNSUPPORTED;
    if (activation < OM_GATE_NONE || activation > OM_GATE_SILU) return OM_ERR_UNSUPPORTED;
    if (!(eps >= 0.0f && eps <= FLT_MAX) || !(fabsf(scale) <= FLT_MAX)) return OM_ERR_INVALID_ARG;
    if (!post && (post_weight || post_bias)) return OM_ERR_INVALID_ARG;
    if (tokens == 0 || width == 0) return OM_OK;
    if (!sum && !out) return OM_ERR_INVALID_ARG;
    if (width > om::kNormMostWidth || tokens > kLim31) return OM_ERR_TOO_LARGE;
    if (!y) return OM_ERR_NULL_PTR;
    // rows of an input may lie in one place (stride 0); an output's may not overlap
    if (ldy < 0 || (residual && ldr < 0) || (gate && ldg < 0)) return OM_ERR_INVALID_ARG;
    if (tokens > 1 && ((sum && lds < width) || (out && ldo < width))) return OM_ERR_INVALID_ARG;
    const int64_t big = int64_t(1) << 40;
    if (ldy > big || (residual && ldr > big) || (gate && ldg > big) || (sum && lds > big) || (out && ldo > big)) return OM_ERR_TOO_LARGE;
    const int64_t tb = type_bytes(dtype), rb = type_bytes(stream_dtype), wb = type_bytes(weight_dtype);
    if (!aligned(y, tb) || !aligned(residual, rb) || !aligned(gate, tb) || !aligned(sum, rb) || !aligned(out, tb) || !aligned(post_weight, wb) ||
        !aligned(post_bias, wb) || !aligned(weight, wb) || !aligned(bias, wb))
        return OM_ERR_ALIGNMENT;
    auto rows = [&](const void *p, int64_t ld, int64_t bytes) { return rows_of(p, tokens, p ? width : 0, ld, bytes); };
    const Block in[7] = {rows(y, ldy, tb), rows(residual, ldr, rb), rows(gate, ldg, tb), rows_of(post_weight, 1, post_weight ? width : 0, 0, wb),
                         rows_of(post_bias, 1, post_bias ? width : 0, 0, wb), rows_of(weight, 1, weight ? width : 0, 0, wb),
                         rows_of(bias, 1, bias ? width : 0, 0, wb)};
    const Block rs = rows(sum, lds, rb), ro = rows(out, ldo, tb);
    if (overlaps(rs, ro)) return OM_ERR_ALIAS;
    // a thread reads its elements of a row before it writes them: an output may take the very place of y or of the residual
    auto one = [&](const void *a, int64_t la, int64_t ba, const void *b, int64_t lb, int64_t bb) { return a == b && ba == bb && (tokens == 1 || la == lb); };
    for (int i = 0; i < 7; ++i) {
        const bool s_here = (i == 0 && one(sum, lds, rb, y, ldy, tb)) || (i == 1 && one(sum, lds, rb, residual, ldr, rb));
        const bool o_here = (i == 0 && one(out, ldo, tb, y, ldy, tb)) || (i == 1 && one(out, ldo, tb, residual, ldr, rb));
        if ((!s_here && overlaps(rs, in[i])) || (!o_here && overlaps(ro, in[i]))) return OM_ERR_ALIAS;
    }
    const om::NormProblem p{tokens, width, y, ldy, dtype, residual, ldr, stream_dtype, gate, ldg, activation, scale, norm == OM_NORM_LAYER, post != 0, eps,
                            post_weight, post_bias, weight, bias, weight_dtype, sum, lds, out, ldo};
    return from_cuda(om::launch_block_norm(p, static_cast<cudaStream_t>(stream)));
}

int om_rope_table(int64_t rows, int64_t rot, double base, int scaling, double factor, double original,
                  double beta_fast, double beta_slow, float *table, void *stream) {
    if (rows < 0 || rot < 2 || rot % 2 != 0 || !(base > 1.0) || !(factor >= 1.0)) return OM_ERR_INVALID_ARG;
    if (scaling < OM_ROPE_PLAIN || scaling > OM_ROPE_YARN) return OM_ERR_UNSUPPORTED;
    if (scaling == OM_ROPE_YARN && !(original > 0.0 && beta_fast > beta_slow && beta_slow > 0.0)) return OM_ERR_INVALID_ARG;
    if (rows > kLim31 || rot > 65536 || rows * (rot / 2) > (int64_t(1) << 37)) return OM_ERR_TOO_LARGE;
    if (rows == 0) return OM_OK;
    if (!table) return OM_ERR_NULL_PTR;
    if (!aligned(table, 4)) return OM_ERR_ALIGNMENT;
    return from_cuda(om::launch_rope_table(rows, rot, base, scaling, factor, original, beta_fast, beta_slow, table,
                                           static_cast<cudaStream_t>(stream)));
}

int om_kv_append_axes(const om_kv_cache *cache, int64_t seqs, int64_t tokens, int64_t max_new, int64_t q_heads,
                 const void *q, int64_t q_ts, int64_t q_hs, const void *k, int64_t k_ts, int64_t k_hs, const void *v,
                 int64_t v_ts, int64_t v_hs, int dtype, const float *table, int64_t rows, int64_t rot, int pairs,
                 const int32_t *block_table, int64_t width, const int32_t *ctx_len, const int32_t *cu, void *q_out,
                 int64_t qo_ts, int64_t qo_hs, const int32_t *positions, int64_t axes, int64_t axis_stride,
                      const int32_t *pair_axis, void *stream) {
    const int cst = check_cache(cache);
    if (cst != OM_OK) return cst;
    const om_kv_cache &c = *cache;
    if (seqs < 0 || tokens < 0 || max_new < 0 || q_heads < 0 || rows < 0) return OM_ERR_INVALID_ARG;
    if (!float_type(dtype)) return OM_ERR_UNSUPPORTED;
    if (rot < 0 || rot > c.dim || (pairs != OM_ROPE_HALF && pairs != OM_ROPE_INTERLEAVED)) return OM_ERR_INVALID_ARG;
    if (rot % 8 != 0) return OM_ERR_UNSUPPORTED;
    if (seqs == 0 || tokens == 0) return OM_OK;
    if (max_new < 1) return OM_ERR_INVALID_ARG;
    const int bst = check_batch(seqs, tokens, block_table, width, c.page, ctx_len, cu);
    if (bst != OM_OK) return bst;
    if (rot > 0 && rows > 0 && !table) return OM_ERR_NULL_PTR;
    if (rows > (int64_t(1) << 40)) return OM_ERR_TOO_LARGE;
    if (!aligned(table, 16)) return OM_ERR_ALIGNMENT;
    if (positions) {
        if (axes < 1 || (axes > 1 && axis_stride < tokens)) return OM_ERR_INVALID_ARG;
        if (axes > 65535 || axis_stride > (int64_t(1) << 40)) return OM_ERR_TOO_LARGE;
    } else if (axes != 0 || pair_axis) {
        return OM_ERR_INVALID_ARG;
    }
    if (!aligned(positions, 4) || !aligned(pair_axis, 4)) return OM_ERR_ALIGNMENT;
    om::KvAppendProblem p{c, seqs, tokens, max_new, q_heads, {q, q_ts, q_hs}, {k, k_ts, k_hs}, {v, v_ts, v_hs},
                          {q_out, qo_ts, qo_hs}, dtype, table, rows, rot, pairs, block_table, width, ctx_len, cu, positions, axes, axis_stride, pair_axis};
    int st = check_heads(p.k, tokens, c.heads, c.dim, dtype, false);
    if (st == OM_OK) st = check_heads(p.v, tokens, c.heads, c.dim, dtype, false);
    if (st == OM_OK && q_heads > 0) st = check_heads(p.q, tokens, q_heads, c.dim, dtype, false);
    if (st == OM_OK && q_heads > 0) st = check_heads(p.q_out, tokens, q_heads, c.dim, dtype, true);
    if (st != OM_OK) return st;
    const int64_t most = max_new < tokens ? max_new : tokens;
    const __int128 blocks = static_cast<__int128>(seqs) * ((most + c.page - 2) / c.page + 1) * c.heads * 2 + tokens;
    if (blocks > kLim31 || q_heads > 65535) return OM_ERR_TOO_LARGE;
    const CacheBlocks cb(c);
    const BatchBlocks bb(seqs, block_table, width, ctx_len, cu);
    const Block rk = heads_block(p.k, tokens, c.heads, c.dim, dtype), rv = heads_block(p.v, tokens, c.heads, c.dim, dtype);
    const Block rt = flat(table, static_cast<__int128>(rows) * rot * 4);
    const Block rp = rows_of(positions, positions ? axes : 0, tokens, axis_stride, 4), ra = flat(pair_axis, pair_axis ? rot / 2 * 4 : 0);
    if (cb.overlap_themselves() || cb.overlap(rk) || cb.overlap(rv) || cb.overlap(rt) || cb.overlap(rp) || cb.overlap(ra)) return OM_ERR_ALIAS;
    for (const Block &x : bb.b)
        if (cb.overlap(x)) return OM_ERR_ALIAS;
    if (q_heads > 0) {
        const Block rq = heads_block(p.q, tokens, q_heads, c.dim, dtype), ro = heads_block(p.q_out, tokens, q_heads, c.dim, dtype);
        if (cb.overlap(rq) || cb.overlap(ro) || overlaps(ro, rk) || overlaps(ro, rv) || overlaps(ro, rt) || overlaps(ro, rp) || overlaps(ro, ra) || bb.overlap(ro) ||
            (!same(p.q, p.q_out) && overlaps(ro, rq)))
            return OM_ERR_ALIAS;
    }
    return from_cuda(om::launch_kv_append(p, static_cast<cudaStream_t>(stream)));
}

int om_kv_append(const om_kv_cache *cache, int64_t seqs, int64_t tokens, int64_t max_new, int64_t q_heads,
                 const void *q, int64_t q_ts, int64_t q_hs, const void *k, int64_t k_ts, int64_t k_hs, const void *v,
                 int64_t v_ts, int64_t v_hs, int dtype, const float *table, int64_t rows, int64_t rot, int pairs,
                 const int32_t *block_table, int64_t width, const int32_t *ctx_len, const int32_t *cu, void *q_out,
                 int64_t qo_ts, int64_t qo_hs, void *stream) {
    return om_kv_append_axes(cache, seqs, tokens, max_new, q_heads, q, q_ts, q_hs, k, k_ts, k_hs, v, v_ts, v_hs, dtype, table, rows, rot, pairs,
                             block_table, width, ctx_len, cu, q_out, qo_ts, qo_hs, nullptr, 0, 0, nullptr, stream);
}

int om_kv_read(const om_kv_cache *cache, int64_t seqs, int64_t tokens, const int32_t *block_table, int64_t width,
               const int32_t *start, const int32_t *cu, void *k_out, void *v_out, int dtype, void *stream) {
    const int cst = check_cache(cache);
    if (cst != OM_OK) return cst;
    const om_kv_cache &c = *cache;
    if (seqs < 0 || tokens < 0) return OM_ERR_INVALID_ARG;
    if (!float_type(dtype)) return OM_ERR_UNSUPPORTED;
    if (seqs == 0 || tokens == 0) return OM_OK;
    const int bst = check_batch(seqs, tokens, block_table, width, c.page, start, cu);
    if (bst != OM_OK) return bst;
    if (!k_out || !v_out) return OM_ERR_NULL_PTR;
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return OM_ERR_ALIGNMENT;
    const __int128 bytes = static_cast<__int128>(tokens) * c.heads * c.dim * type_bytes(dtype);
    const Block rk = flat(k_out, bytes), rv = flat(v_out, bytes);
    const CacheBlocks cb(c);
    const BatchBlocks bb(seqs, block_table, width, start, cu);
    if (overlaps(rk, rv) || cb.overlap(rk) || cb.overlap(rv) || bb.overlap(rk) || bb.overlap(rv)) return OM_ERR_ALIAS;
    const om::KvReadProblem p{c, seqs, tokens, block_table, width, start, cu, k_out, v_out, dtype};
    return from_cuda(om::launch_kv_read(p, static_cast<cudaStream_t>(stream)));
}

size_t om_kv_workspace_bytes(int64_t kv_heads, int64_t q_heads, int64_t dim, int64_t max_new) {
    if (kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 || dim < 1 || max_new < 1 || dim > 65536) return 0;
    return om::kv_workspace_bytes(q_heads / kv_heads, dim, max_new);
}

int om_kv_attention_sinks(const om_kv_cache *cache, int64_t seqs, int64_t tokens, int64_t max_new, int64_t q_heads,
                          const void *q, int64_t q_ts, int64_t q_hs, int dtype, const int32_t *block_table, int64_t width,
                          const int32_t *ctx_len, const int32_t *cu, float scale, int64_t window, int64_t sinks, void *out,
                          int64_t o_ts, int64_t o_hs, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    const int cst = check_cache(cache);
    if (cst != OM_OK) return cst;
    const om_kv_cache &c = *cache;
    if (seqs < 0 || tokens < 0 || max_new < 0 || q_heads < 1 || window < 0 || sinks < 0) return OM_ERR_INVALID_ARG;
    if (q_heads % c.heads != 0) return OM_ERR_INVALID_ARG;
    if (!float_type(dtype)) return OM_ERR_UNSUPPORTED;
    if (seqs == 0 || tokens == 0) return OM_OK;
    if (max_new < 1) return OM_ERR_INVALID_ARG;
    const int bst = check_batch(seqs, tokens, block_table, width, c.page, ctx_len, cu);
    if (bst != OM_OK) return bst;
    if (q_heads > 65535 || tokens * q_heads > kLim31 - kMargin) return OM_ERR_TOO_LARGE;
    // pieces of 64 positions of every key head and eight query rows, at most
    const __int128 units = static_cast<__int128>(width * c.page / 64 + 1) * c.heads * (tokens * (q_heads / c.heads) / 8 + seqs);
    if (units > kLim31 - (1 << 20)) return OM_ERR_TOO_LARGE;
    // a window of all positions there can be is none (the kernel takes positions less the window in 64 bits), and so is one beside first
    // positions that are all the table has
    const bool bound = window > 0 && window < kLim31 && sinks < width * c.page;
    om::KvAttentionProblem p{c, seqs, tokens, max_new, q_heads, {q, q_ts, q_hs}, {out, o_ts, o_hs}, dtype, lse,
                             block_table, width, ctx_len, cu, scale, bound ? window : 0, workspace, bound ? static_cast<int>(sinks) : 0};
    int st = check_heads(p.q, tokens, q_heads, c.dim, dtype, false);
    if (st == OM_OK) st = check_heads(p.out, tokens, q_heads, c.dim, dtype, true);
    if (st != OM_OK) return st;
    if (!aligned(lse, 4)) return OM_ERR_ALIGNMENT;
    if (workspace) {
        if (!aligned(workspace, 16)) return OM_ERR_ALIGNMENT;
        if (workspace_bytes < om::kv_workspace_bytes(q_heads / c.heads, c.dim, max_new)) return OM_ERR_INVALID_ARG;
    }
    const CacheBlocks cb(c);
    const BatchBlocks bb(seqs, block_table, width, ctx_len, cu);
    const Block rq = heads_block(p.q, tokens, q_heads, c.dim, dtype);
    const Block w[3] = {heads_block(p.out, tokens, q_heads, c.dim, dtype),
                        flat(lse, lse ? static_cast<__int128>(tokens) * q_heads * 4 : 0),
                        flat(workspace, workspace ? static_cast<__int128>(workspace_bytes) : 0)};
    for (int i = 0; i < 3; ++i) {
        if (cb.overlap(w[i]) || bb.overlap(w[i]) || overlaps(w[i], rq)) return OM_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(w[i], w[j])) return OM_ERR_ALIAS;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == OM_F32) return from_cuda(p.sinks > 0 ? om::launch_kv_attention_sinks_f32(p, s) : om::launch_kv_attention_f32(p, s));
    if (dtype == OM_F16) return from_cuda(p.sinks > 0 ? om::launch_kv_attention_sinks_f16(p, s) : om::launch_kv_attention_f16(p, s));
    return from_cuda(p.sinks > 0 ? om::launch_kv_attention_sinks_bf16(p, s) : om::launch_kv_attention_bf16(p, s));
}

int om_kv_attention(const om_kv_cache *cache, int64_t seqs, int64_t tokens, int64_t max_new, int64_t q_heads,
                    const void *q, int64_t q_ts, int64_t q_hs, int dtype, const int32_t *block_table, int64_t width,
                    const int32_t *ctx_len, const int32_t *cu, float scale, int64_t window, void *out, int64_t o_ts,
                    int64_t o_hs, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    return om_kv_attention_sinks(cache, seqs, tokens, max_new, q_heads, q, q_ts, q_hs, dtype, block_table, width, ctx_len, cu, scale, window, 0, out,
                                 o_ts, o_hs, lse, workspace, workspace_bytes, stream);
}

size_t om_kv_shared_workspace_bytes(int64_t kv_heads, int64_t q_heads, int64_t dim, int64_t max_new, int64_t tokens) {
    if (kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 || dim < 1 || max_new < 1 || dim > 65536 || tokens < 1) return 0;
    if (q_heads > 65535 || tokens > kLim31 / q_heads) return 0;
    return shared_places(nullptr, q_heads / kv_heads, q_heads, dim, max_new, tokens).bytes;
}

int om_kv_shared_attention(const om_kv_cache *cache, int64_t groups, const int32_t *prefix_table, int64_t prefix_width, const int32_t *prefix_len,
                           const int32_t *group_offsets, int64_t seqs, int64_t tokens, int64_t max_new, int64_t q_heads, const void *q, int64_t q_ts,
                           int64_t q_hs, int dtype, const int32_t *block_table, int64_t width, const int32_t *ctx_len, const int32_t *cu, float scale,
                           void *out, int64_t o_ts, int64_t o_hs, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    const int cst = check_cache(cache);
    if (cst != OM_OK) return cst;
    const om_kv_cache &c = *cache;
    if (groups < 0 || seqs < 0 || tokens < 0 || max_new < 0 || q_heads < 1 || q_heads % c.heads != 0) return OM_ERR_INVALID_ARG;
    if (!float_type(dtype)) return OM_ERR_UNSUPPORTED;
    if (seqs == 0 || tokens == 0) return OM_OK;
    if (max_new < 1) return OM_ERR_INVALID_ARG;
    int st = check_batch(seqs, tokens, block_table, width, c.page, ctx_len, cu);
    if (st == OM_OK && groups > 0) st = check_batch(groups, tokens, prefix_table, prefix_width, c.page, prefix_len, group_offsets);
    if (st != OM_OK) return st;
    if (q_heads > 65535 || tokens * q_heads > kLim31 - kMargin) return OM_ERR_TOO_LARGE;
    const int64_t group = q_heads / c.heads;
    // pieces of 64 positions of every key head and eight query rows, at most
    const __int128 units = static_cast<__int128>(width * c.page / 64 + 1) * c.heads * (tokens * group / 8 + seqs);
    // and of the prefixes, for every 128 rows
    const __int128 prefix_units = groups > 0 ? static_cast<__int128>(prefix_width * c.page / 64 + 1) * c.heads * (tokens * group / om::kSharedRows + groups) : 0;
    if (units > kLim31 - (1 << 20) || prefix_units > kLim31 - (1 << 21)) return OM_ERR_TOO_LARGE;
    const Heads hq{q, q_ts, q_hs}, ho{out, o_ts, o_hs};
    st = check_heads(hq, tokens, q_heads, c.dim, dtype, false);
    if (st == OM_OK) st = check_heads(ho, tokens, q_heads, c.dim, dtype, true);
    if (st != OM_OK) return st;
    if (!workspace) return OM_ERR_NULL_PTR;
    if (!aligned(lse, 4) || !aligned(workspace, 16)) return OM_ERR_ALIGNMENT;
    const SharedPlaces at = shared_places(workspace, group, q_heads, c.dim, max_new, tokens);
    if (workspace_bytes < at.bytes) return OM_ERR_INVALID_ARG;
    const CacheBlocks cb(c);
    const BatchBlocks bb(seqs, block_table, width, ctx_len, cu), pb(groups, prefix_table, prefix_width, prefix_len, groups > 0 ? group_offsets : cu);
    const Block rq = heads_block(hq, tokens, q_heads, c.dim, dtype);
    const Block w[3] = {heads_block(ho, tokens, q_heads, c.dim, dtype), flat(lse, lse ? static_cast<__int128>(tokens) * q_heads * 4 : 0),
                        flat(workspace, static_cast<__int128>(workspace_bytes))};
    for (int i = 0; i < 3; ++i) {
        if (cb.overlap(w[i]) || bb.overlap(w[i]) || (groups > 0 && pb.overlap(w[i])) || overlaps(w[i], rq)) return OM_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(w[i], w[j])) return OM_ERR_ALIAS;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int64_t blocks = static_cast<int64_t>(om::num_sms()) * (c.dim == 256 ? 1 : 2);
    if (blocks > om::kSharedMostBlocks) blocks = om::kSharedMostBlocks;
    if (prefix_units < blocks) blocks = static_cast<int64_t>(prefix_units);
    if (blocks < 1) blocks = 1;
    const int64_t eb = type_bytes(dtype);
    om::SharedProblem p{};
    p.c = c;
    p.seqs = seqs; p.tokens = tokens; p.q_heads = q_heads; p.groups = groups;
    p.q = hq;
    p.dtype = dtype;
    p.group = static_cast<int>(group);
    p.q_sixteens = aligned(q, 16) && q_ts * eb % 16 == 0 && q_hs * eb % 16 == 0;
    p.prefix_table = prefix_table; p.prefix_width = prefix_width; p.prefix_len = prefix_len; p.group_at = group_offsets; p.cu = cu;
    p.scale = scale;
    p.blocks = blocks;
    p.most_tiles = groups < 1 ? 0 : std::min(prefix_width * c.page / om::kSharedTile + 1, static_cast<int64_t>(prefix_units) / blocks + 1);
    p.slot_rows = at.slot_rows;
    p.whole_state = at.whole_state; p.slot_state = at.slot_state; p.whole = at.whole; p.slots = at.slots; p.kept = at.kept;
    p.own_state = at.own_state; p.own = at.own;
    p.out = ho;
    p.lse = lse;
    p.status = static_cast<unsigned *>(workspace) + om::kWsStatusWord;
    if (groups > 0) {
        const bool pages = c.page < om::kSharedTile;
        const cudaError_t e = c.dtype == OM_I8 ? (pages ? om::launch_kv_shared_pages_i8(p, s) : om::launch_kv_shared_i8(p, s))
                                               : (pages ? om::launch_kv_shared_pages_e4m3(p, s) : om::launch_kv_shared_e4m3(p, s));
        if (e != cudaSuccess) return OM_ERR_CUDA;
    }
    const om::KvAttentionProblem own{c, seqs, tokens, max_new, q_heads, hq, {at.own, q_heads * c.dim, c.dim}, dtype, reinterpret_cast<float *>(at.own_state),
                                     block_table, width, ctx_len, cu, scale, 0, workspace, 0};
    const cudaError_t e = dtype == OM_F32 ? om::launch_kv_attention_part_f32(own, s)
                          : dtype == OM_F16 ? om::launch_kv_attention_part_f16(own, s) : om::launch_kv_attention_part_bf16(own, s);
    if (e != cudaSuccess) return OM_ERR_CUDA;
    return from_cuda(om::launch_kv_shared_join(p, s));
}

}  // extern "C"
