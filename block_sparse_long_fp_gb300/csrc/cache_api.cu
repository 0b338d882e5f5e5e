// The C ABI of the bf16 / e4m3 paged cache and of rotary positions: argument checks and
// launches.
#include <math.h>
#include <string.h>

#include "cache.cuh"

using namespace fp;

namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

fp_status check_ws(const void *ws, size_t ws_bytes) {
    if (!ws || ws_bytes < FP_WS_HEADER_BYTES) return FP_ERR_WORKSPACE;
    return aligned(ws, 4) ? FP_OK : FP_ERR_INVALID;
}

bool dtype_ok(fp_dtype t) { return t == FP_BF16 || t == FP_E4M3; }

// Rows of `heads` vectors of kHeadDim elements that do not overlap, 16-byte aligned; an e4m3
// row has a scale a head.
bool rows_ok(const void *p, long long tok, long long head, int heads, fp_dtype t, const float *scale) {
    const int esz = t == FP_E4M3 ? 1 : 2;
    const long long most = 1ll << 38;          // what the copies' descriptors take
    return p && aligned(p, 16) && head >= kHeadDim && head <= most && tok <= most &&
           tok >= head * (heads - 1) + kHeadDim && (tok * esz) % 16 == 0 && (head * esz) % 16 == 0 &&
           (t == FP_BF16 || (scale && aligned(scale, 4)));
}

fp_status check_rope(const fp_rope_table *t, bool inverse, Rotation *rot) {
    if (!t || t->rot < 2 || t->rot > kHeadDim || t->rot % 2) return FP_ERR_INVALID;
    if (t->layout != FP_ROPE_HALF && t->layout != FP_ROPE_INTERLEAVED) return FP_ERR_INVALID;
    if (!t->turns || !aligned(t->turns, 8) || !isfinite(t->scale)) return FP_ERR_INVALID;
    *rot = Rotation{t->turns, t->rot, t->layout == FP_ROPE_INTERLEAVED, t->scale, inverse ? -t->scale : t->scale};
    return FP_OK;
}

// What this build supports of a cache's shape.
fp_status check_shape(const fp_cache *c) {
    if (c->d != kHeadDim) return FP_ERR_UNSUPPORTED;
    if (c->page_size < 16 || !(kBlock % c->page_size == 0 || c->page_size % kBlock == 0)) return FP_ERR_UNSUPPORTED;
    return (long long)c->num_pages * c->page_size > (1ll << 31) - 1 ? FP_ERR_UNSUPPORTED : FP_OK;
}

fp_status check_cache(const fp_cache *c) {
    if (!c || c->h_kv < 1 || c->num_pages < 1 || !dtype_ok(c->dtype)) return FP_ERR_INVALID;
    const fp_status s = check_shape(c);
    if (s != FP_OK) return s;
    const long long tok = (long long)c->h_kv * kHeadDim;
    if (!rows_ok(c->k, tok, kHeadDim, c->h_kv, c->dtype, c->k_scale) ||
        !rows_ok(c->v, tok, kHeadDim, c->h_kv, c->dtype, c->v_scale))
        return FP_ERR_INVALID;
    return FP_OK;
}

// Heads and rows that a launch can count.
bool countable(long long rows, long long heads) { return rows <= 1 << 30 && heads <= 1 << 16 && rows * heads <= 1ll << 33; }

RowsPart part(const void *in, long long in_tok, long long in_head, void *out, long long out_tok, long long out_head,
              int heads, fp_dtype t, const float *scale) {
    return RowsPart{static_cast<const __nv_bfloat16 *>(in), out, in_tok, in_head, out_tok, out_head,
                    t == FP_E4M3 ? scale : nullptr, heads};
}

// Everything of an attention call but its buffers.
fp_status check_query(const fp_cache *c, const fp_qcache_query *q, PAttn *a) {
    if (!c || c->h_kv < 1 || c->num_pages < 1 || !dtype_ok(c->dtype)) return FP_ERR_INVALID;
    const fp_status s = check_shape(c);
    if (s != FP_OK) return s;
    if (!q || q->batch < 1 || q->total_q < 0 || q->max_q < 1 || q->max_pages_per_seq < 1) return FP_ERR_INVALID;
    if (q->batch > FP_TABLES_MAX_BATCH) return FP_ERR_UNSUPPORTED;
    if (q->h_q < 1 || q->h_q % c->h_kv || !dtype_ok(q->dtype)) return FP_ERR_INVALID;
    if ((long long)q->total_q * q->h_q > (1ll << 30)) return FP_ERR_UNSUPPORTED;
    if (!q->cu_seqlens_q && (long long)q->batch * q->max_q > q->total_q) return FP_ERR_INVALID;
    memset(a, 0, sizeof(*a));
    a->c = Pages{static_cast<const unsigned char *>(c->k), static_cast<const unsigned char *>(c->v), c->num_pages,
                 c->page_size, c->h_kv};
    a->k_scale = c->dtype == FP_E4M3 ? c->k_scale : nullptr;
    a->v_scale = c->dtype == FP_E4M3 ? c->v_scale : nullptr;
    a->batch = q->batch;
    a->h_q = q->h_q;
    a->g = q->h_q / c->h_kv;
    a->total_q = q->total_q;
    a->max_q = q->max_q;
    a->q = q->q;
    a->q_stride_tok = q->q_stride_tok;
    a->q_stride_head = q->q_stride_head;
    a->q_scale = q->dtype == FP_E4M3 ? q->q_scale : nullptr;
    a->q_codes = q->dtype == FP_E4M3;
    a->cu = q->cu_seqlens_q;
    a->seqlens_k = q->seqlens_k;
    a->block_table = q->block_table;
    a->max_pages = q->max_pages_per_seq;
    const long long held = (long long)q->max_pages_per_seq * c->page_size, most = (1ll << 31) - 64;
    a->max_len = (int)(held < most ? held : most);
    a->scale = q->softmax_scale > 0.f ? q->softmax_scale : 1.f / sqrtf((float)kHeadDim);
    return FP_OK;
}

}  // namespace

extern "C" {

fp_status fp_rope_turns(const double *inv_freq, int n, unsigned long long *turns) {
    if (!inv_freq || !turns || n < 1) return FP_ERR_INVALID;
    for (int i = 0; i < n; ++i)
        if (!(fabs(inv_freq[i]) <= 0x1p20)) return FP_ERR_INVALID;
    for (int i = 0; i < n; ++i) {
        // a double's quotient has 53 right bits: its remainder, divided too, gives the rest
        const double pi_hi = 0x1.921fb54442d18p+2, pi_lo = 0x1.1a62633145c07p-52;     // 2 pi in two terms
        const double f = fabs(inv_freq[i]), hi = f / pi_hi;
        const double lo = (fma(-hi, pi_hi, f) - hi * pi_lo) / pi_hi;
        const double frac = hi - floor(hi);                                           // exact
        // in two halves, as frac 2^64 is past what converts to an integer
        const double upper = floor(frac * 0x1p32), rest = (frac * 0x1p32 - upper) * 0x1p32;
        const unsigned long long low = (unsigned long long)(long long)rint(rest + lo * 0x1p64);
        const unsigned long long x = ((unsigned long long)upper << 32) + low;
        turns[i] = inv_freq[i] < 0 ? 0 - x : x;
    }
    return FP_OK;
}

fp_status fp_rope(const fp_rope_table *t, const fp_rope_rows *r, void *stream) {
    RotateRows a;
    memset(&a, 0, sizeof(a));
    if (!r || r->rows < 0 || r->heads < 1 || !dtype_ok(r->out_dtype) || (r->inverse != 0 && r->inverse != 1))
        return FP_ERR_INVALID;
    const fp_status s = check_rope(t, r->inverse != 0, &a.rot);
    if (s != FP_OK) return s;
    if (!countable(r->rows, r->heads)) return FP_ERR_UNSUPPORTED;
    if (r->rows == 0) return FP_OK;
    if (!r->positions || !aligned(r->positions, 4) ||
        !rows_ok(r->x, r->x_stride_tok, r->x_stride_head, r->heads, FP_BF16, nullptr) ||
        !rows_ok(r->out, r->out_stride_tok, r->out_stride_head, r->heads, r->out_dtype, r->out_scale))
        return FP_ERR_INVALID;
    a.positions = r->positions;
    a.rows = r->rows;
    a.q = part(r->x, r->x_stride_tok, r->x_stride_head, r->out, r->out_stride_tok, r->out_stride_head, r->heads,
               r->out_dtype, r->out_scale);
    return launch_rotate_rows(a, (cudaStream_t)stream) == cudaSuccess ? FP_OK : FP_ERR_CUDA;
}

fp_status fp_cache_append(const fp_cache *c, const fp_rope_table *rope_opt, const fp_cache_rows *r, void *ws,
                          size_t ws_bytes, void *stream) {
    RotateRows a;
    memset(&a, 0, sizeof(a));
    fp_status s = check_cache(c);
    if (s != FP_OK) return s;
    if (!r || r->rows < 0 || r->h_q < 0 || (r->q == nullptr) != (r->h_q == 0)) return FP_ERR_INVALID;
    if (rope_opt && (s = check_rope(rope_opt, false, &a.rot)) != FP_OK) return s;
    if (!countable(r->rows, (long long)r->h_q + 2 * (long long)c->h_kv)) return FP_ERR_UNSUPPORTED;
    if (r->q && !dtype_ok(r->q_dtype)) return FP_ERR_INVALID;
    if (r->rows > 0) {
        if (!r->slots || !aligned(r->slots, 4) || (rope_opt && (!r->positions || !aligned(r->positions, 4))) ||
            !rows_ok(r->k, r->k_stride_tok, r->k_stride_head, c->h_kv, FP_BF16, nullptr) ||
            !rows_ok(r->v, r->v_stride_tok, r->v_stride_head, c->h_kv, FP_BF16, nullptr))
            return FP_ERR_INVALID;
        if (r->q && (!rows_ok(r->q, r->q_stride_tok, r->q_stride_head, r->h_q, FP_BF16, nullptr) ||
                     !rows_ok(r->q_out, r->q_out_stride_tok, r->q_out_stride_head, r->h_q, r->q_dtype, r->q_scale)))
            return FP_ERR_INVALID;
    }
    if ((s = check_ws(ws, ws_bytes)) != FP_OK) return s;
    if (r->rows == 0) return FP_OK;
    const long long tok = (long long)c->h_kv * kHeadDim;
    a.positions = rope_opt ? r->positions : nullptr;
    a.rows = r->rows;
    if (r->q)
        a.q = part(r->q, r->q_stride_tok, r->q_stride_head, r->q_out, r->q_out_stride_tok, r->q_out_stride_head, r->h_q,
                   r->q_dtype, r->q_scale);
    a.k = part(r->k, r->k_stride_tok, r->k_stride_head, c->k, tok, kHeadDim, c->h_kv, c->dtype, c->k_scale);
    a.v = part(r->v, r->v_stride_tok, r->v_stride_head, c->v, tok, kHeadDim, c->h_kv, c->dtype, c->v_scale);
    a.slots = r->slots;
    a.num_slots = (long long)c->num_pages * c->page_size;
    a.status = static_cast<int *>(ws);
    return launch_rotate_rows(a, (cudaStream_t)stream) == cudaSuccess ? FP_OK : FP_ERR_CUDA;
}

size_t fp_cache_attn_scratch_bytes(const fp_cache *c, const fp_qcache_query *q) {
    PAttn a;
    if (check_query(c, q, &a) != FP_OK) return 0;
    a.k_scale = c->dtype == FP_E4M3 ? reinterpret_cast<const float *>(16) : nullptr;     // the type alone counts
    return cache_attn_scratch_bytes(a);
}

fp_status fp_cache_attn(const fp_cache *c, const fp_qcache_query *q, void *out, float *lse_opt, void *scratch,
                        size_t scratch_bytes, void *ws, size_t ws_bytes, void *stream) {
    PAttn a;
    fp_status s = check_query(c, q, &a);
    if (s != FP_OK || (s = check_cache(c)) != FP_OK) return s;
    if (!q->seqlens_k || !q->block_table || !aligned(q->seqlens_k, 4) || !aligned(q->block_table, 4) ||
        !aligned(q->cu_seqlens_q, 4))
        return FP_ERR_INVALID;
    if (q->total_q > 0) {
        if (!out || !aligned(out, 16) || !aligned(lse_opt, 4)) return FP_ERR_INVALID;
        if (!rows_ok(q->q, q->q_stride_tok, q->q_stride_head, q->h_q, q->dtype, q->q_scale)) return FP_ERR_INVALID;
    }
    if ((s = check_ws(ws, ws_bytes)) != FP_OK) return s;
    if (!scratch || !aligned(scratch, 16) || scratch_bytes < cache_attn_scratch_bytes(a)) return FP_ERR_WORKSPACE;
    if (q->total_q == 0) return FP_OK;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse_opt;
    a.status = static_cast<int *>(ws);
    return launch_cache_attn(a, scratch, wait_limit_ns(), (cudaStream_t)stream) == cudaSuccess ? FP_OK : FP_ERR_CUDA;
}

}  // extern "C"
