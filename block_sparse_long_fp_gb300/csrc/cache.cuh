// The bf16 / e4m3 paged K/V cache and rotary positions as their kernels see them.
#pragma once

#include <atomic>

#include "qcache.cuh"

namespace fp {

struct Rotation {
    const unsigned long long *turns;           // [rot / 2]; null: none
    int rot;
    bool interleaved;
    float scale;                               // of cos, and of sin (negated there for the inverse)
    float sin_scale;
};

// `heads` vectors of kHeadDim elements a row: bf16 in, bf16 or (with scales) e4m3 out.
struct RowsPart {
    const __nv_bfloat16 *in;
    void *out;
    long long in_tok, in_head, out_tok, out_head;   // elements
    const float *scale;
    int heads;
};

struct RotateRows {
    Rotation rot;
    const int *positions;                      // null: nothing is rotated
    int rows;
    RowsPart q, k, v;                          // q and k are rotated; k and v go to row slots[i]
    const int *slots;
    long long num_slots;
    int *status;
};
cudaError_t launch_rotate_rows(const RotateRows &r, cudaStream_t st);

struct Pages {
    const unsigned char *k, *v;                // [num_pages, page_size, h_kv, kHeadDim]
    int num_pages, page_size, h_kv;
};

struct PAttn {
    Pages c;
    const float *k_scale, *v_scale;            // null for bf16
    int batch, h_q, g, total_q, max_q;
    const void *q;
    long long q_stride_tok, q_stride_head;
    const float *q_scale;                      // null for bf16
    const int *cu;                             // null: max_q rows each
    const int *seqlens_k, *block_table;
    int max_pages;
    int max_len;                               // what the table holds, short of what an int's arithmetic can
    float scale;                               // logit scale
    __nv_bfloat16 *out;
    float *lse;
    int *status;
    bool whole;                                // no item is cut (set by the launch)
    bool q_codes;                              // e4m3 queries
    int half;                                  // queries of half a tile (set by the launch)
    const signed char *q_exponent;             // of the power of two of converted bf16 queries (set by the launch)
    int most_columns;                          // rows times g up to which a request is the columns' (set by the launch)
};
// cache_attn.cu: by columns, and which of the two takes what
size_t cache_attn_scratch_bytes(const PAttn &a);
cudaError_t launch_cache_attn(const PAttn &a, void *scratch, unsigned long long limit_ns, cudaStream_t st);
// cache_tiles.cu: the requests of more columns, by tiles
size_t cache_tiles_scratch_bytes(const PAttn &a);
cudaError_t launch_cache_tiles(const PAttn &a, void *scratch, unsigned long long limit_ns, cudaStream_t st);
// the limit of bounded waits (fp_set_wait_limit_ns)
unsigned long long wait_limit_ns();

// A launch with more shared memory than the default limit, which a kernel is given once on
// each device (it takes as long as the launch).  A device that was reset since is told again.
template <typename... P, typename... A>
cudaError_t launch_large(std::atomic<unsigned long long> &told, void (*kernel)(P...), unsigned grid, unsigned block, int smem,
                         cudaStream_t st, A... args) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = device < 64 ? 1ull << device : 0;
    const bool known = told.load(std::memory_order_relaxed) & bit;
    for (int attempt = known ? 0 : 1; attempt < 2; ++attempt) {
        if (attempt) {
            if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
            told.fetch_or(bit, std::memory_order_relaxed);
        }
        e = launch_chained(kernel, grid, block, (size_t)smem, st, args...);
        if (e != cudaErrorInvalidValue || attempt) return e;
        cudaGetLastError();
    }
    return e;
}

}  // namespace fp
