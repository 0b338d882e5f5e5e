// The C ABI of the serving operators (page tables, the 4-bit cache, attention
// over it): argument checks and launches.
#include <math.h>
#include <string.h>

#include "qcache.cuh"

using namespace fp;

namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int *status_of(void *ws) { return static_cast<int *>(ws); }

fp_status check_pages(int page_size, int num_pages) {
    if (page_size < 16 || !((kBlock % page_size == 0) || (page_size % kBlock == 0))) return FP_ERR_UNSUPPORTED;
    if (num_pages < 1) return FP_ERR_INVALID;
    return (long long)num_pages * page_size > (1ll << 31) - 1 ? FP_ERR_UNSUPPORTED : FP_OK;
}

fp_status check_ws(const void *ws, size_t ws_bytes) {
    if (!ws || ws_bytes < FP_WS_HEADER_BYTES) return FP_ERR_WORKSPACE;
    return aligned(ws, 4) ? FP_OK : FP_ERR_INVALID;
}

// The shape of a cache, without its data.
fp_status check_shape(const fp_qcache *c) {
    if (!c || c->h_kv < 1) return FP_ERR_INVALID;
    if (c->d != kHeadDim) return FP_ERR_UNSUPPORTED;
    if (c->group != 32 && c->group != 64 && c->group != 128) return FP_ERR_UNSUPPORTED;
    return check_pages(c->page_size, c->num_pages);
}

fp_status view(const fp_qcache *c, QCache *out) {
    const fp_status s = check_shape(c);
    if (s != FP_OK) return s;
    if (!c->data || !aligned(c->data, 16)) return FP_ERR_INVALID;
    *out = QCache{static_cast<unsigned char *>(c->data), c->num_pages, c->page_size, c->h_kv, kHeadDim / c->group};
    return FP_OK;
}

// Rows of `heads` vectors of kHeadDim elements that do not overlap, 16-byte aligned.
bool strides_ok(long long tok, long long head, int heads, int esz) {
    return head >= kHeadDim && tok >= head * (heads - 1) + kHeadDim && (tok * esz) % 16 == 0 && (head * esz) % 16 == 0;
}

fp_status check_rows(const fp_qcache *c, const fp_qcache_rows *r, bool read, QCache *cache, QRows *rows) {
    fp_status s = view(c, cache);
    if (s != FP_OK) return s;
    if (!r || r->rows < 0) return FP_ERR_INVALID;
    if (r->dtype != FP_BF16 && r->dtype != FP_E4M3) return FP_ERR_INVALID;
    if (r->rows == 0) {
        rows->rows = 0;
        return FP_OK;
    }
    if (!r->k || !r->v || !r->slots || !aligned(r->k, 16) || !aligned(r->v, 16)) return FP_ERR_INVALID;
    if (!aligned(r->slots, 4) || !aligned(r->out_slots, 4)) return FP_ERR_INVALID;
    if (!strides_ok(r->stride_tok, r->stride_head, c->h_kv, r->dtype == FP_E4M3 ? 1 : 2)) return FP_ERR_INVALID;
    if (r->dtype == FP_E4M3 && (!r->k_scale || !r->v_scale || !aligned(r->k_scale, 4) || !aligned(r->v_scale, 4)))
        return FP_ERR_INVALID;
    if (read && (r->out_rows < 0 || (!r->out_slots && r->out_rows < r->rows))) return FP_ERR_INVALID;
    if (r->rows > (1 << 30) || (long long)r->rows * c->h_kv > (1ll << 33)) return FP_ERR_UNSUPPORTED;
    *rows = QRows{r->k, r->v, r->stride_tok, r->stride_head, r->slots, read ? r->out_slots : nullptr, r->rows,
                  r->out_rows, r->dtype == FP_E4M3 ? r->k_scale : nullptr, r->dtype == FP_E4M3 ? r->v_scale : nullptr};
    return FP_OK;
}

// Everything of an attention call but its buffers.
fp_status check_query(const fp_qcache *c, const fp_qcache_query *q, QAttn *a) {
    fp_status s = check_shape(c);
    if (s != FP_OK) return s;
    if (!q || q->batch < 1 || q->total_q < 0 || q->max_q < 1 || q->max_pages_per_seq < 1) return FP_ERR_INVALID;
    if (q->batch > FP_TABLES_MAX_BATCH) return FP_ERR_UNSUPPORTED;
    if (q->h_q < 1 || q->h_q % c->h_kv) return FP_ERR_INVALID;
    if (q->dtype != FP_BF16 && q->dtype != FP_E4M3) return FP_ERR_INVALID;
    if ((long long)q->total_q * q->h_q > (1ll << 30)) return FP_ERR_UNSUPPORTED;
    if (!q->cu_seqlens_q && (long long)q->batch * q->max_q > q->total_q) return FP_ERR_INVALID;
    memset(a, 0, sizeof(*a));
    a->c = QCache{static_cast<unsigned char *>(c->data), c->num_pages, c->page_size, c->h_kv, kHeadDim / c->group};
    a->batch = q->batch;
    a->h_q = q->h_q;
    a->g = q->h_q / c->h_kv;
    a->total_q = q->total_q;
    a->max_q = q->max_q;
    a->q = q->q;
    a->q_stride_tok = q->q_stride_tok;
    a->q_stride_head = q->q_stride_head;
    a->q_scale = q->dtype == FP_E4M3 ? q->q_scale : nullptr;
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

size_t fp_qcache_chunk_bytes(const fp_qcache *c) {
    return check_shape(c) == FP_OK ? qcache_chunk_bytes(kHeadDim / c->group) : 0;
}

size_t fp_qcache_bytes(const fp_qcache *c) {
    if (check_shape(c) != FP_OK) return 0;
    return (size_t)c->num_pages * c->h_kv * (c->page_size / kChunk) * qcache_chunk_bytes(kHeadDim / c->group);
}

fp_status fp_page_tables(const fp_tables *t, void *ws, size_t ws_bytes, void *stream) {
    if (!t || t->batch < 1 || t->max_pages_per_seq < 1 || t->num_free < 0 || t->capacity < 1) return FP_ERR_INVALID;
    if (t->batch > FP_TABLES_MAX_BATCH) return FP_ERR_UNSUPPORTED;
    fp_status s = check_pages(t->page_size, t->num_pages);
    if (s != FP_OK) return s;
    if (!t->seqlens || !t->new_lens || (!t->free_pages && t->num_free) || !t->block_table || !t->cu_seqlens_q ||
        !t->seqlens_k || !t->positions || !t->slots || !t->free_next)
        return FP_ERR_INVALID;
    if (!aligned(t->positions, 16) || !aligned(t->slots, 16)) return FP_ERR_INVALID;
    for (const void *p : {(const void *)t->seqlens, (const void *)t->new_lens, (const void *)t->free_pages,
                          (const void *)t->free_head, (const void *)t->block_table, (const void *)t->cu_seqlens_q,
                          (const void *)t->seqlens_k, (const void *)t->free_next})
        if (!aligned(p, 4)) return FP_ERR_INVALID;
    if ((s = check_ws(ws, ws_bytes)) != FP_OK) return s;
    return launch_page_tables(*t, status_of(ws), (cudaStream_t)stream) == cudaSuccess ? FP_OK : FP_ERR_CUDA;
}

fp_status fp_qcache_write(const fp_qcache *c, const fp_qcache_rows *r, void *ws, size_t ws_bytes, void *stream) {
    QCache cache;
    QRows rows;
    fp_status s = check_rows(c, r, false, &cache, &rows);
    if (s != FP_OK || (s = check_ws(ws, ws_bytes)) != FP_OK) return s;
    if (rows.rows == 0) return FP_OK;
    return launch_qcache_write(cache, rows, rows.k_scale != nullptr, status_of(ws), (cudaStream_t)stream) == cudaSuccess
               ? FP_OK
               : FP_ERR_CUDA;
}

fp_status fp_qcache_read(const fp_qcache *c, const fp_qcache_rows *r, void *ws, size_t ws_bytes, void *stream) {
    QCache cache;
    QRows rows;
    fp_status s = check_rows(c, r, true, &cache, &rows);
    if (s != FP_OK || (s = check_ws(ws, ws_bytes)) != FP_OK) return s;
    if (rows.rows == 0) return FP_OK;
    return launch_qcache_read(cache, rows, rows.k_scale != nullptr, status_of(ws), (cudaStream_t)stream) == cudaSuccess
               ? FP_OK
               : FP_ERR_CUDA;
}

size_t fp_qcache_attn_scratch_bytes(const fp_qcache *c, const fp_qcache_query *q) {
    QAttn a;
    return check_query(c, q, &a) == FP_OK ? qcache_attn_scratch_bytes(a) : 0;
}

fp_status fp_qcache_attn(const fp_qcache *c, const fp_qcache_query *q, void *out, float *lse_opt, void *scratch,
                         size_t scratch_bytes, void *ws, size_t ws_bytes, void *stream) {
    QAttn a;
    fp_status s = check_query(c, q, &a);
    if (s != FP_OK) return s;
    if (!c->data || !aligned(c->data, 16)) return FP_ERR_INVALID;
    if (!q->seqlens_k || !q->block_table || !aligned(q->seqlens_k, 4) || !aligned(q->block_table, 4) ||
        !aligned(q->cu_seqlens_q, 4))
        return FP_ERR_INVALID;
    if (q->total_q > 0) {
        if (!q->q || !aligned(q->q, 16) || !out || !aligned(out, 16) || !aligned(lse_opt, 4)) return FP_ERR_INVALID;
        if (!strides_ok(q->q_stride_tok, q->q_stride_head, q->h_q, q->dtype == FP_E4M3 ? 1 : 2)) return FP_ERR_INVALID;
        if (q->dtype == FP_E4M3 && (!q->q_scale || !aligned(q->q_scale, 4))) return FP_ERR_INVALID;
    }
    if ((s = check_ws(ws, ws_bytes)) != FP_OK) return s;
    if (!scratch || !aligned(scratch, 16) || scratch_bytes < qcache_attn_scratch_bytes(a)) return FP_ERR_WORKSPACE;
    if (q->total_q == 0) return FP_OK;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse_opt;
    a.status = status_of(ws);
    return launch_qcache_attn(a, scratch, (cudaStream_t)stream) == cudaSuccess ? FP_OK : FP_ERR_CUDA;
}

}  // extern "C"
