// The 4-bit K/V cache as its kernels see it: addresses inside the chunk layout
// that fprefill.h documents, and the launch interface.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace fp {

constexpr int kChunk = 16;                     // tokens of a chunk
constexpr int kCodeBytes = kChunk * kHeadDim / 2;   // K codes (or V codes) of a chunk

struct QCache {
    unsigned char *data;
    int num_pages, page_size, h_kv, groups;    // groups: 128 / group
};

__host__ __device__ __forceinline__ int qcache_chunk_bytes(int groups) { return 2 * kCodeBytes + 128 * groups; }

// The chunk that holds `slot` of `head`; offsets pass 32 bits in a long cache.
__device__ __forceinline__ unsigned char *qcache_chunk(const QCache &c, int slot, int head) {
    const int page = slot / c.page_size, off = slot - page * c.page_size;
    const long long chunk = ((long long)page * c.h_kv + head) * (c.page_size / kChunk) + off / kChunk;
    return c.data + chunk * qcache_chunk_bytes(c.groups);
}

// Byte offsets inside a chunk.  K and V codes: the 2 bytes that hold dims
// 4 l .. 4 l + 3 of token t.  The f16 arrays: the step of token t, group g (the
// minimum is 32 * groups bytes behind it).
__device__ __forceinline__ int k_code_off(int t, int l) { return t * 64 + ((l & 7) >> 1) * 16 + (l >> 3) * 4 + (l & 1) * 2; }
__device__ __forceinline__ int v_code_off(int t, int l) {
    return kCodeBytes + (t >> 3) * 512 + (l & 7) * 64 + ((t & 7) >> 1) * 16 + (t & 1) * 8 + (l >> 3) * 2;
}
__device__ __forceinline__ int k_step_off(int t, int g, int groups) { return 2 * kCodeBytes + (t * groups + g) * 2; }
__device__ __forceinline__ int v_step_off(int t, int g, int groups) {
    return 2 * kCodeBytes + 64 * groups + ((((t & 7) >> 1) * groups + g) * 4 + (t >> 3) * 2 + (t & 1)) * 2;
}

// Launches that are set up while the kernel before them in the stream ends, which hides
// some of a launch's latency in a chain of short kernels: every kernel here waits for the
// one before (after_previous) before it touches memory.  A kernel may also let the next
// one's blocks onto the SMs while it runs itself (let_next): there they wait, and hold what
// they were given, so only a short one at the end of a call does (256 requests up to 2048
// tokens: 99 us when the attention did, 78 us without).
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Two fp32 in one register pair, each rounded by itself.
using float_pair = unsigned long long;
__device__ __forceinline__ float_pair pair(float lo, float hi) {
    float_pair y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(lo), "f"(hi));
    return y;
}
__device__ __forceinline__ float2 unpair(float_pair x) {
    float2 y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(x));
    return y;
}
__device__ __forceinline__ float_pair fma2(float_pair a, float_pair b, float_pair c) {
    float_pair y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
    return y;
}
__device__ __forceinline__ float_pair add2(float_pair a, float_pair b) {
    float_pair y;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}
__device__ __forceinline__ float_pair mul2(float_pair a, float_pair b) {
    float_pair y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}
struct QRows {
    const void *k, *v;
    long long stride_tok, stride_head;
    const int *slots, *out_slots;
    int rows, out_rows;
    const float *k_scale, *v_scale;            // null for bf16
};
cudaError_t launch_qcache_write(const QCache &c, const QRows &r, bool fp8, int *status, cudaStream_t st);
cudaError_t launch_qcache_read(const QCache &c, const QRows &r, bool fp8, int *status, cudaStream_t st);

struct QAttn {
    QCache c;
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
};
size_t qcache_attn_scratch_bytes(const QAttn &a);
cudaError_t launch_qcache_attn(const QAttn &a, void *scratch, cudaStream_t st);

cudaError_t launch_page_tables(const fp_tables &t, int *status, cudaStream_t st);

}  // namespace fp
