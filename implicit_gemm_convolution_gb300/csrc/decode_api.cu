// decode_api.cu -- the C ABI of the decoding operators: argument validation and launch
// on the caller's stream. Nothing is launched by a call that fails validation.
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

int om_kv_append(const om_kv_cache *cache, int64_t seqs, int64_t tokens, int64_t max_new, int64_t q_heads,
                 const void *q, int64_t q_ts, int64_t q_hs, const void *k, int64_t k_ts, int64_t k_hs, const void *v,
                 int64_t v_ts, int64_t v_hs, int dtype, const float *table, int64_t rows, int64_t rot, int pairs,
                 const int32_t *block_table, int64_t width, const int32_t *ctx_len, const int32_t *cu, void *q_out,
                 int64_t qo_ts, int64_t qo_hs, void *stream) {
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
    om::KvAppendProblem p{c, seqs, tokens, max_new, q_heads, {q, q_ts, q_hs}, {k, k_ts, k_hs}, {v, v_ts, v_hs},
                          {q_out, qo_ts, qo_hs}, dtype, table, rows, rot, pairs, block_table, width, ctx_len, cu};
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
    if (cb.overlap_themselves() || cb.overlap(rk) || cb.overlap(rv) || cb.overlap(rt)) return OM_ERR_ALIAS;
    for (const Block &x : bb.b)
        if (cb.overlap(x)) return OM_ERR_ALIAS;
    if (q_heads > 0) {
        const Block rq = heads_block(p.q, tokens, q_heads, c.dim, dtype), ro = heads_block(p.q_out, tokens, q_heads, c.dim, dtype);
        if (cb.overlap(rq) || cb.overlap(ro) || overlaps(ro, rk) || overlaps(ro, rv) || overlaps(ro, rt) || bb.overlap(ro) ||
            (!same(p.q, p.q_out) && overlaps(ro, rq)))
            return OM_ERR_ALIAS;
    }
    return from_cuda(om::launch_kv_append(p, static_cast<cudaStream_t>(stream)));
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

int om_kv_attention(const om_kv_cache *cache, int64_t seqs, int64_t tokens, int64_t max_new, int64_t q_heads,
                    const void *q, int64_t q_ts, int64_t q_hs, int dtype, const int32_t *block_table, int64_t width,
                    const int32_t *ctx_len, const int32_t *cu, float scale, int64_t window, void *out, int64_t o_ts,
                    int64_t o_hs, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    const int cst = check_cache(cache);
    if (cst != OM_OK) return cst;
    const om_kv_cache &c = *cache;
    if (seqs < 0 || tokens < 0 || max_new < 0 || q_heads < 1 || window < 0) return OM_ERR_INVALID_ARG;
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
    // a window of all positions there can be is none: the kernel takes positions less the window in 64 bits
    om::KvAttentionProblem p{c, seqs, tokens, max_new, q_heads, {q, q_ts, q_hs}, {out, o_ts, o_hs}, dtype, lse,
                             block_table, width, ctx_len, cu, scale, window < kLim31 ? window : 0, workspace};
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
    if (dtype == OM_F32) return from_cuda(om::launch_kv_attention_f32(p, s));
    return from_cuda(dtype == OM_F16 ? om::launch_kv_attention_f16(p, s) : om::launch_kv_attention_bf16(p, s));
}

}  // extern "C"
