// What the attentions over device lengths share (the 4-bit cache's and the bf16 / e4m3
// one's): requests as the kernels read them, the items' scan, asynchronous copies, and the
// join of items that several thread blocks share.  `A` is the arguments' structure (QAttn,
// PAttn), which name these fields alike.
#pragma once

#include <cuda_fp16.h>

#include "qcache.cuh"

namespace fp {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSm = 152;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTop = 10.f, kSlack = 4.f;   // log2 of the largest weight, where its maximum is set and where it follows
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kOutStride = kHeadDim + 4;     // floats per column of a warp's result in shared memory

// An item that its first thread block leaves open: where, and in how many parts.
struct __align__(16) Open {
    int parts, row0, rows, kv, tile, pad[3];
};

struct Scratch {
    Open *open;                              // [blocks]
    float2 *ml;                              // [blocks][2][cols]: exponent base and weight sum
    float *o;                                // [blocks][2][cols][kHeadDim]
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// The base that a largest logit of m sets: kTop below it; m itself from 2^27 on, where fp32's neighbours are 16
// and more apart and m - kTop would round to m - 16, which makes a weight that fp16 does not hold.
__device__ __forceinline__ float base_below(float m) {
    const float b = m - kTop;
    return m - b <= kTop + kSlack ? b : m;
}

// Transpose of the 8 x 8 fp16 matrix whose row lane / 4 holds the lane's pair.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

struct Request {
    int row0, lq, rows, len;      // rows: those of its lq that q has
};

template <typename A>
__device__ __forceinline__ Request request_of(const A &a, int r) {
    Request q;
    if (a.cu) {
        const int x = a.cu[r], y = a.cu[r + 1];
        q.row0 = x;
        q.lq = x >= 0 && y > x ? y - x : 0;
        q.rows = min(q.lq, max(0, a.total_q - x));
        if (x < 0 || q.rows < q.lq) set_status(a.status, FP_ERR_DEVICE_BOUNDS);
    } else {
        q.row0 = r * a.max_q;
        q.lq = q.rows = a.max_q;
    }
    q.len = a.seqlens_k[r];
    if (q.len < 0 || q.len > a.max_len) {
        set_status(a.status, FP_ERR_DEVICE_BOUNDS);
        q.len = 0;
    }
    return q;
}
template <typename A>
__device__ __forceinline__ int tiles_of(const A &a, const Request &q, int cols) {
    return (int)(((long long)q.rows * a.g + cols - 1) / cols);
}
// Chunks of an item; an empty cache counts as one, which writes its zeros.
__device__ __forceinline__ int chunks_of(const Request &q) { return q.len > 0 ? (q.len + kChunk - 1) / kChunk : 1; }

// O = v / l and its log-sum-exp, top + log2(l) in base 2; zeros and -inf without a key.
template <typename A>
__device__ __forceinline__ void store_row(const A &a, int row, int head, int lane, float4 v, float top, float l) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat162 x = __floats2bfloat162_rn(v.x * inv, v.y * inv), y = __floats2bfloat162_rn(v.z * inv, v.w * inv);
    *reinterpret_cast<uint2 *>(a.out + ((long long)row * a.h_q + head) * kHeadDim + 4 * lane) =
        make_uint2(*reinterpret_cast<uint32_t *>(&x), *reinterpret_cast<uint32_t *>(&y));
    if (a.lse && lane == 0) a.lse[(long long)head * a.total_q + row] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
}

// Exclusive scan over the block; *all is the sum.
__device__ __forceinline__ long long block_scan(long long n, long long *all, long long *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    long long x = n;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const long long y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    long long sum = 0;
    x -= n;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const long long v = warp_sums[w];
        if (w < warp) x += v;
        sum += v;
    }
    __syncthreads();
    *all = sum;
    return x;
}

// a / b of two that are not negative.  A division of 64 bits is a call of some 100
// dependent instructions, and a block's start would have six of them.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// Joins the parts of the items that several blocks share: part 0 in the first
// block's second slot, the others in the first slots of the blocks behind it.
// A task is a column of an open item.  With 8 parts and more to an item a block
// takes a task, its warps a share of the parts each; else a warp does.
constexpr int kJoinWarps = 8;

// kMost: blocks at most.
template <int NT, int kMost, typename A>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(A a, Scratch sc, int blocks) {
    constexpr int kCols = 8 * NT;
    constexpr int kEach = (kMost + kJoinWarps * 32 - 1) / (kJoinWarps * 32);
    __shared__ Open list[kMost];
    __shared__ int first[kMost], count[kEach][kJoinWarps];
    __shared__ float4 part_o[kJoinWarps][32];
    __shared__ float part_l[kJoinWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    after_previous();
    let_next();
    // the items that blocks left open, in the same order for every block of this grid
    Open rec[kEach];
    unsigned vote[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int b = e * kJoinWarps * 32 + threadIdx.x;
        rec[e].parts = 0;
        if (b < blocks) rec[e] = sc.open[b];
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        vote[e] = __ballot_sync(~0u, rec[e].parts > 0);
        if (lane == 0) count[e][warp] = __popc(vote[e]);
    }
    __syncthreads();
    int opens = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        int at = opens + __popc(vote[e] & ((1u << lane) - 1));
        for (int w = 0; w < kJoinWarps; ++w) {
            if (w < warp) at += count[e][w];
            opens += count[e][w];
        }
        if (rec[e].parts > 0) {
            list[at] = rec[e];
            first[at] = e * kJoinWarps * 32 + threadIdx.x;
        }
    }
    __syncthreads();
    const bool wide = opens * 8 <= blocks;
    const int step = wide ? 1 : kJoinWarps, w0 = wide ? warp : 0, dw = wide ? kJoinWarps : 1;
    for (int task0 = blockIdx.x * step; task0 < opens * kCols; task0 += gridDim.x * step) {
        const int task = task0 + (wide ? 0 : warp);
        const bool live = task < opens * kCols;
        const int b = first[live ? task / kCols : 0], col = task % kCols;
        const Open it = list[live ? task / kCols : 0];
        const int cc = it.tile * kCols + col, i = cc / a.g, head = it.kv * a.g + cc % a.g;
        float top = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live && i < it.rows) {
            const auto slot = [&](int p) { return ((long long)(b + p) * 2 + (p == 0)) * kCols + col; };
            for (int p = lane; p < it.parts; p += 32) top = fmaxf(top, sc.ml[slot(p)].x);
#pragma unroll
            for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
#pragma unroll 4
            for (int p = w0; p < it.parts; p += dw) {
                const float2 e = sc.ml[slot(p)];
                const float4 v = *reinterpret_cast<const float4 *>(sc.o + slot(p) * kHeadDim + 4 * lane);
                const float f = e.x == -INFINITY ? 0.f : exp2f(e.x - top);
                l += e.x == -INFINITY ? e.y : f * e.y;
                o.x = fmaf(f, v.x, o.x);
                o.y = fmaf(f, v.y, o.y);
                o.z = fmaf(f, v.z, o.z);
                o.w = fmaf(f, v.w, o.w);
            }
            if (!wide) store_row(a, it.row0 + i, head, lane, o, top, l);
        }
        if (wide) {
            part_o[warp][lane] = o;
            if (lane == 0) part_l[warp] = l;
            __syncthreads();
            if (warp == 0 && i < it.rows) {
                for (int w = 1; w < kJoinWarps; ++w) {
                    const float4 v = part_o[w][lane];
                    l += part_l[w];
                    o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
                }
                store_row(a, it.row0 + i, head, lane, o, top, l);
            }
            __syncthreads();
        }
    }
}

constexpr size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace
}  // namespace fp
