// The bf16 / e4m3 paged K/V cache and rotary positions as their kernels see them.
#pragma once

#include <cuda_fp16.h>

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
// a wait of the tiles on a barrier that nothing arrives on (fp_check_wait_timeout)
cudaError_t launch_cache_wait_timeout(int *status, unsigned long long limit_ns, cudaStream_t st);
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

// Two e4m3 codes in the low half of a register, as fp16.
__device__ __forceinline__ uint32_t halves_of(uint32_t codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3);
    return (uint32_t)h.x | (uint32_t)h.y << 16;
}
// Two numbers as fp16 (of an e4m3 cache) or bf16.
template <bool kFp8>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if (kFp8) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Two e4m3 codes as bf16, which holds them.
__device__ __forceinline__ uint32_t bf16_of(uint32_t codes) {
    const uint32_t h = halves_of(codes);
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack16<false>(v.x, v.y);
}
// Two elements of a bf16 query for an e4m3 cache: times `up`, a power of two that brings the row's largest
// into [2^7, 2^8), each as two e4m3 codes of 4 bits, which hold 8 bits exactly down to 2^-9 of the largest, and
// the rest to 2^-17 of it.
struct TwoTerms {
    uint32_t hi, lo;
};
__device__ __forceinline__ TwoTerms two_terms(float a, float b, float up) {
    // an infinity becomes a NaN: e4m3 would take it for its largest value
    const float x = fmaf(a, up, a * 0.f), y = fmaf(b, up, b * 0.f);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3), back = halves_of(hi);
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&back));
    return {hi, __nv_cvt_float2_to_fp8x2(make_float2(x - v.x, y - v.y), __NV_SATFINITE, __NV_E4M3)};
}
__device__ __forceinline__ int term_exp(float top) { return fp16_scale_exp(__float_as_uint(top)) - 7; }

}  // namespace fp
