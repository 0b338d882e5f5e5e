// fp_qcache_attn: attention over the 4-bit cache.
//
// Arithmetic.  A nibble c in the low ten bits of an fp16 is the subnormal
// c 2^-24 (or c 2^-20 four bits up), exactly, and the tensor cores multiply
// subnormals at full rate.  So the codes go into m16n8k16 products as they lie
// in memory, one AND a pair, and steps and minima fold in around them:
//   K: S^T[token, col] = sum_g s_g(t) (C_g Q^T)[t, col] + (M Qsum^T)[t, col]
//      -- a product per group of dims, its fp32 result times the token's step,
//      plus one m16n8k8 product of the minima with the queries' group sums (two
//      fp16 terms each); dims whose nibble lies four bits up meet queries / 16.
//   V: O^T[dim, col] = sum_t c_g(t) (p_t s_g(t)), the weights times the steps
//      rounded to fp16 as the B operand, plus one product of the minima with
//      the weights; rows whose nibble lies four bits up end 16 times too large.
// A column is one (query, head) of the kv head's group, so the keys fill the
// long side of the instruction and 8 columns suffice for a decode step: with
// tokens on the short side half of every instruction would be padding.
// Queries enter as fp16 under a power of two per row (exact for bf16 and e4m3
// within 2^-29 of the row's largest), logits, weights' sums and outputs are fp32 (a
// chunk's products join them by an addition of their own), weights are fp16 (2^-11 each,
// as is their product with a step).
//
// Weights are exp2(logit - m + 10), m a maximum that only follows when the logits pass
// it by 4 (a warp vote), so that the largest weight so far is between 2^10 and 2^14.  V
// steps meet them times a power of two of their group, which sums take back at the item's
// end and which only falls: where a step times it would reach 2, it is set anew, to bring
// the group's largest of that chunk to 2^-2 .. 2^-1 (steps of 2 and more to 1 .. 2, as they
// are few and the others' lose bits below 2^-14), and the group's sums with it.  Weight
// times step stays below 2^15, and fp16 flushes weights below 2^-35 of the largest, and
// products below 2^-33 of the largest weight times its group's largest step, whatever the
// steps of the other groups are.
//
// Work.  The (request, kv head, column tile) items laid end to end, each as long as its
// start and end cost plus its chunks of 16 tokens, are cut into equal ranges, one per
// thread block, whatever the lengths (which only the GPU knows).  The warps of a block take
// every kWarps-th chunk of an item, each through a ring of its own in shared memory
// (cp.async: nothing to wait on but its own copies), and join their results at the item's
// end.  An item cut by a range's end leaves partial results, which a second kernel joins, in
// a fixed order: the same call gives the same bits.
//
// Bounds.  One octet of columns: memory, with about 295 instructions a chunk (88 of them
// take codes apart) that leave little slack: 64 requests of up to 16384 tokens (32/4 heads,
// groups of 32) 63 us, one of 262144 (32/8) 62 us, 5.3 TB/s each, 0.78 of the measured copy
// rate; 4 us of it pass before the first chunk and 4 in the join.  More octets: each adds
// about 100 instructions a chunk, and a warp's instructions follow each other at 4 to 8 cycles
// whatever the occupancy that the registers leave.  16 columns (4 tokens of 4 heads) over 32
// requests of 4096 on average: 55 us, 32 columns: 94 us, where the products alone need 33.
#include <limits.h>

#include <type_traits>

#include "qcache.cuh"

namespace fp {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSm = 152;
constexpr int kMinChunks = 2 * kWarps;       // least work worth a thread block
// Work is cut in units.  What starting and ending an item costs, in chunks, and what a
// chunk costs by the octets of columns in use (extracting the codes is most of it; with
// one octet at most there is nothing to tell apart).
template <int NT>
constexpr int item_chunks() { return NT == 1 ? 24 : NT == 2 ? 28 : 40; }
template <int NT>
__device__ __forceinline__ int chunk_units(int octets) { return NT == 1 ? 1 : 2 + octets; }
// Longest cache, by the width of its table, that is not cut (one launch instead of two).
// Microseconds whole / cut, 32/8 heads, with 8, 16, 32 columns, tables filled:
//   up to 1024, 1 request    10.9 /  8.2   16.3 / 10.6   23.2 / 16.2
//               16           11.0 / 13.2   16.7 / 17.7   23.0 / 26.9
//               64           22.7 / 24.2   35.9 / 37.6   55.0 / 62.9
//   up to 2048, 1            17.1 /  9.0   26.0 / 11.3   35.4 / 15.5
//               16           17.2 / 16.1   26.3 / 21.9   36.2 / 35.2
// and filled to 0.3:
//   up to 1024, 1             6.9 /  8.0    9.8 /  9.9   13.4 / 15.6
//   up to 2048, 1             8.8 /  8.3   12.8 / 10.4   17.2 / 14.5
constexpr int kWholeChunks = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTop = 10.f, kSlack = 4.f;   // log2 of the largest weight, where its maximum is set and where it follows
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kOutStride = kHeadDim + 4;     // floats per column of a warp's result in shared memory

// An item that its first thread block leaves open: where, and in how many parts.
struct __align__(16) Open {
    int parts, row0, rows, kv, tile, pad[3];
};

// What a page id out of range, or an empty cache, reads.
__device__ __align__(16) unsigned char zero_chunk[2 * kCodeBytes + 128 * 4];

struct Scratch {
    Open *open;                              // [blocks]
    float2 *ml;                              // [blocks][2][cols]: exponent base and weight sum
    float *o;                                // [blocks][2][cols][kHeadDim]
};

// Blocks per SM, by their registers (168 a thread for 3, 255 for 2), and copies ahead.  8
// columns, 64 requests up to 16384 tokens / one of 262144 / 256 up to 2048: 62 / 61 / 77 us;
// with 4 blocks 66 / 66 / 77, with 2 68 / 63 / 107, with 3 and 6 copies 65 / 64 / 79.  16
// columns, 32 requests up to 8192: 55 us; with 4 blocks, which spill, 61, with 2 58.
template <int NT>
constexpr int blocks_per_sm() { return NT == 1 ? 3 : NT == 2 ? 3 : 2; }
template <int NT>
constexpr int stages() { return NT == 4 ? 8 : 4; }

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mma16(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero: the accumulator needs no clearing.
__device__ __forceinline__ void mma16_zero(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma8_zero(float d[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
// Sums over the length are added in fp32, rounded to nearest: chained on the tensor cores,
// which cut the bits below their largest term off, they lose some 2^-25 of themselves a
// product, always towards zero.  Codes are positive and minima make up for it, so that the
// outputs of 262144 tokens in one block, of values of zero mean, were off by 0.023 of
// themselves, and are by 0.002 now, the output's own rounding.
__device__ __forceinline__ void add_to(float &a, float &b, float x, float y) {
    const float2 v = unpair(add2(pair(a, b), pair(x, y)));
    a = v.x;
    b = v.y;
}
// Transpose of the 8 x 8 fp16 matrix whose row lane / 4 holds the lane's pair.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    const __half2 h = __hmul2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&h);
}
// The exponent of a power of two in fp16 (both halves alike), and the pair of one.
__device__ __forceinline__ int exponent_of(uint32_t x) {
    return (__float_as_int(__half2float(__ushort_as_half((unsigned short)x))) >> 23) - 127;
}
__device__ __forceinline__ uint32_t power_pair(int e) { return pack_half2(pow2f(e), pow2f(e)); }
__device__ __forceinline__ uint32_t shared_word(uint32_t at) {
    uint32_t x;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(at));
    return x;
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

__device__ __forceinline__ Request request_of(const QAttn &a, int r) {
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
__device__ __forceinline__ int tiles_of(const QAttn &a, const Request &q, int cols) {
    return (int)(((long long)q.rows * a.g + cols - 1) / cols);
}
// Chunks of an item; an empty cache counts as one, which writes its zeros.
__device__ __forceinline__ int chunks_of(const Request &q) { return q.len > 0 ? (q.len + kChunk - 1) / kChunk : 1; }

// O = v / l and its log-sum-exp, top + log2(l) in base 2; zeros and -inf without a key.
__device__ __forceinline__ void store_row(const QAttn &a, int row, int head, int lane, float4 v, float top, float l) {
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

// The operands that one lane holds for 8 columns: queries as B fragments
// ([quarter of the dims][half of its 16 bytes] of (b0, b1)), the query's sum over
// group lane % 4 times 2^-18 in two fp16 terms, and what a column's fp32 products
// times 2^24 have to be scaled by to be base-2 logits.
struct Queries {
    uint2 f[4][2];
    uint32_t sum;
    float factor;      // of column lane / 4
};

// A column's 32 elements of this lane as they lie in memory (bf16, or e4m3 in the
// first half), and its scale.
struct RawQuery {
    uint4 w[4];
    float scale;
};

__device__ __forceinline__ RawQuery fetch_query(const QAttn &a, const Request &q, int kv, int col) {
    const int j4 = threadIdx.x & 3, i = col / a.g, head = kv * a.g + col % a.g;
    RawQuery raw;
    raw.scale = a.scale * kLog2e;
#pragma unroll
    for (int y = 0; y < 4; ++y) raw.w[y] = make_uint4(0, 0, 0, 0);
    if (i < q.rows) {
        const long long at = (q.row0 + i) * a.q_stride_tok + head * a.q_stride_head + 8 * j4;
        if (a.q_scale) {
            raw.scale *= a.q_scale[head];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const unsigned char *>(a.q) + at + 32 * y);
                raw.w[y].x = w.x;
                raw.w[y].y = w.y;
            }
        } else {
#pragma unroll
            for (int y = 0; y < 4; ++y)
                raw.w[y] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + at + 32 * y);
        }
    }
    return raw;
}

template <int NG>
__device__ __forceinline__ void make_queries(const RawQuery &raw, bool fp8, Queries &out) {
    const int j4 = threadIdx.x & 3;
    float x[32], top = 0.f, f = raw.scale;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        const uint32_t v[4] = {raw.w[y].x, raw.w[y].y, raw.w[y].z, raw.w[y].w};
        if (fp8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                __nv_fp8_e4m3 c;
                c.__x = (__nv_fp8_storage_t)((v[e / 4] >> (8 * (e & 3))) & 0xff);
                x[8 * y + e] = (float)c;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[8 * y + 2 * e] = __uint_as_float(v[e] << 16);
                x[8 * y + 2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) top = fmaxf(top, fabsf(x[e]));
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
    const int ex = fp16_scale_exp(__float_as_uint(top));
    const float up = pow2f(ex);
    float gs = 0.f;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        float part = 0.f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float *p = x + 8 * y + 2 * u;
            const __half2 b0 = __floats2half2_rn(p[0] * up, p[4] * up);
            const __half2 b1 = __floats2half2_rn(p[1] * up * 0.0625f, p[5] * up * 0.0625f);
            out.f[y][u] = make_uint2(*reinterpret_cast<const uint32_t *>(&b0), *reinterpret_cast<const uint32_t *>(&b1));
            const float2 f0 = __half22float2(b0), f1 = __half22float2(b1);
            part += f0.x + f0.y + 16.f * (f1.x + f1.y);
        }
        part += __shfl_xor_sync(~0u, part, 1);
        part += __shfl_xor_sync(~0u, part, 2);
        gs += y * NG / 4 == j4 ? part : 0.f;
    }
    gs *= 0x1p-18f;
    const float hi = __half2float(__float2half_rn(gs));
    out.sum = pack_half2(hi, gs - hi);
    out.factor = f * pow2f(24) * pow2f(-ex);
}

// NG fp16 from shared memory, as floats.
template <int NG>
__device__ __forceinline__ void load_halves(const unsigned char *p, float out[NG]) {
    if (NG == 4) {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
        out[0] = a.x, out[1 % NG] = a.y, out[2 % NG] = b.x, out[3 % NG] = b.y;
    } else if (NG == 2) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(p));
        out[0] = a.x, out[1 % NG] = a.y;
    } else {
        out[0] = __half2float(*reinterpret_cast<const __half *>(p));
    }
}

// a / b of two that are not negative.  A division of 64 bits is a call of some 100
// dependent instructions, and a block's start would have six of them.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

template <int NG, int NT>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<NT>()) attn_kernel(QAttn a, Scratch sc) {
    constexpr int kCols = 8 * NT, kBytes = 2 * kCodeBytes + 128 * NG, kStages = stages<NT>();
    constexpr int kRing = kStages * kBytes, kItem = item_chunks<NT>();
    constexpr bool kSharedQ = NT > 1;          // queries' fragments in shared memory instead of registers
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ long long warp_sums[kWarps];
    __shared__ long long s_at;
    __shared__ int s_r;
    __shared__ Request s_q;
    __shared__ float2 ml[kWarps][kCols];
    __shared__ uint2 s_frag[kSharedQ ? NT : 1][4][2][32];
    __shared__ uint32_t s_sum[kSharedQ ? NT : 1][32];
    __shared__ float s_factor[kSharedQ ? kCols : 1];
    after_previous();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31, r8 = lane >> 2, j4 = lane & 3;

    // this block's range of units, and the request it starts in: an item is its start and
    // end, then its chunks
    const auto octets_of = [&](const Request &q, int tile) { return (min(kCols, q.rows * a.g - tile * kCols) + 7) / 8; };
    const auto units = [&](const Request &q) {
        const int tiles = tiles_of(a, q, kCols);
        if (tiles == 0 || a.whole) return (long long)a.c.h_kv * tiles;
        return (long long)a.c.h_kv * (kItem + chunks_of(q)) *
               ((tiles - 1) * chunk_units<NT>(NT) + chunk_units<NT>(octets_of(q, tiles - 1)));
    };
    const int each = (a.batch + kThreads - 1) / kThreads;      // requests a thread adds up
    Request q = {0, 0, 0, 0};
    long long n = 0, total;
    for (int r = tid * each; r < min(a.batch, (tid + 1) * each); ++r) n += units(q = request_of(a, r));
    long long low = block_scan(n, &total, warp_sums);
    const long long want = a.whole ? total : total / (kMinChunks * chunk_units<NT>(NT)) + 1;
    const int blocks = total == 0 ? 0 : (int)(want < gridDim.x ? want : gridDim.x);
    if (tid == 0 && !a.whole) sc.open[blockIdx.x].parts = 0;
    if ((int)blockIdx.x >= blocks) return;
    // the first `longer` blocks have `share` + 1 units, the others `share`
    const long long share = quotient(total, blocks);
    const int longer = (int)(total - share * blocks);
    const long long first = blockIdx.x * share + min((int)blockIdx.x, longer), end = first + share + ((int)blockIdx.x < longer);
    if (low <= first && first < low + n) {
        int r = tid * each;
        if (each > 1)
            for (;; ++r) {
                n = units(q = request_of(a, r));
                if (first < low + n || r + 1 == a.batch) break;
                low += n;
            }
        s_r = r;
        s_at = low;
        s_q = q;
    }
    __syncthreads();
    int r = s_r;
    long long item0 = s_at;                       // first unit of the current item
    q = s_q;
    int tiles = tiles_of(a, q, kCols), chunks = chunks_of(q);
    int kv, tile;                                 // of the current item
    {
        const long long full = a.whole ? 1 : (long long)(kItem + chunks) * chunk_units<NT>(NT);
        const long long last = a.whole ? 1 : (long long)(kItem + chunks) * chunk_units<NT>(octets_of(q, tiles - 1));
        const long long head = (tiles - 1) * full + last;
        kv = (int)quotient(first - item0, head);
        item0 += kv * head;
        tile = min((int)quotient(first - item0, full), tiles - 1);
        item0 += tile * full;
    }
    unsigned char *ring = smem + warp * kRing;
    const uint32_t ring_at = smem_addr(ring) + lane * 16;
    const int per_page = a.c.page_size / kChunk;

    for (long long at = first; at < end;) {
        if (tile == tiles) {
            tile = 0;
            ++kv;
        }
        while (kv >= a.c.h_kv || tiles == 0) {    // the next request that has rows
            if (++r >= a.batch) return;           // lengths that changed under the kernel
            q = request_of(a, r);
            tiles = tiles_of(a, q, kCols);
            chunks = chunks_of(q);
            kv = tile = 0;
        }
        const int octets = octets_of(q, tile), weight = chunk_units<NT>(octets);
        const long long next = a.whole ? item0 + 1 : item0 + (long long)(kItem + chunks) * weight;
        const int c0 = a.whole ? 0 : max(0, (int)((uint32_t)(at - item0) / weight) - kItem);    // an item is below 2^30 units
        const int c1 = a.whole ? chunks : max(0, (int)((uint32_t)(min(end, next) - item0) / weight) - kItem);
        if (c1 <= c0) {                           // the range ends inside the item's start
            at = item0 = next;
            ++tile;
            continue;
        }
        const int mine = c1 - c0 > warp ? (c1 - c0 - warp + kWarps - 1) / kWarps : 0;

        // -- copies ahead: chunk c0 + warp + i * kWarps into stage i % kStages.  Lane l
        //    looks up the addresses of chunks l, l + 32, ...
        unsigned long long src = 0;
        int page = -1, in_page = 0;
        const auto look_up = [&](int i) {         // the page id of chunk i + lane ...
            const int c = c0 + warp + (i + lane) * kWarps, pg = c / per_page;
            page = i + lane < mine && q.len > 0 ? a.block_table[(long long)r * a.max_pages + pg] : -1;
            in_page = c - pg * per_page;
        };
        const auto locate = [&](int i) {          // ... and the chunk's address
            src = (unsigned long long)zero_chunk;
            if (page >= 0 && page < a.c.num_pages)
                src = (unsigned long long)(a.c.data + (((long long)page * a.c.h_kv + kv) * per_page + in_page) * kBytes);
            else if (i + lane < mine && q.len > 0)
                set_status(a.status, FP_ERR_DEVICE_BOUNDS);
        };
        int issued = 0;
        const auto issue = [&]() {
            if (issued < mine) {
                if (issued && issued % 32 == 0) {
                    look_up(issued);
                    locate(issued);
                }
                const unsigned long long from = __shfl_sync(~0u, src, issued & 31);
                const uint32_t dst = ring_at + (issued % kStages) * kBytes;
                const char *p = reinterpret_cast<const char *>(from) + lane * 16;
#pragma unroll
                for (int i = 0; i < (kBytes + 511) / 512; ++i)
                    if ((i + 1) * 512 <= kBytes || lane * 16 < kBytes - i * 512) copy16(dst + i * 512, p + i * 512);
                ++issued;
            }
            copies_commit();
        };
        look_up(0);

        // -- queries of this item: their loads go out before the page ids arrive ------
        constexpr int kOwn = kSharedQ ? (NT + kWarps - 1) / kWarps : NT;       // column octets this warp prepares
        RawQuery raw[kOwn];
#pragma unroll
        for (int t = 0; t < kOwn; ++t) {
            const int octet = kSharedQ ? t * kWarps + warp : t;
            if (octet < NT) raw[t] = fetch_query(a, q, kv, tile * kCols + octet * 8 + r8);
        }
        locate(0);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue();
        Queries qs[kOwn];
#pragma unroll
        for (int t = 0; t < kOwn; ++t) {
            const int octet = kSharedQ ? t * kWarps + warp : t;
            if (octet >= NT) continue;            // whole warps
            make_queries<NG>(raw[t], a.q_scale != nullptr, qs[t]);
            if (kSharedQ) {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    s_frag[octet][y][0][lane] = qs[t].f[y][0];
                    s_frag[octet][y][1][lane] = qs[t].f[y][1];
                }
                s_sum[octet][lane] = qs[t].sum;
                if (j4 == 0) s_factor[octet * 8 + r8] = qs[t].factor;
            }
        }
        if (kSharedQ) __syncthreads();
        float factor[NT][2];
        const int min_keys = min(q.len, q.len - q.lq + tile * kCols / a.g + 1);     // of the tile's first query
        // keys that column c of this lane (of 8 t + 2 j4 + e) may see
        const auto keys_of = [&](int t, int e) {
            const int i = (tile * kCols + t * 8 + 2 * j4 + e) / a.g;
            return min(q.len, q.len - q.lq + i + 1);
        };
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                factor[t][e] = kSharedQ ? s_factor[t * 8 + 2 * j4 + e]
                                        : __shfl_sync(~0u, qs[kSharedQ ? 0 : t].factor, (2 * j4 + e) * 4);

        float o[NT][8][4];                        // O^T: 8 tiles of 16 dims
        float z[NT][2];                           // the minima's part, a row per group
        float base[NT][2];                        // log2 of what weight 1 stands for (-inf: no key yet)
        float sum[NT][2];                         // this lane's share of the weights
        uint32_t up[NG];                          // what a group's V steps are multiplied by, as a pair
#pragma unroll
        for (int g = 0; g < NG; ++g) up[g] = 0x78007800u;             // 2^15
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int m = 0; m < 8; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][m][e] = 0.f;
            z[t][0] = z[t][1] = 0.f;
            base[t][0] = base[t][1] = -INFINITY;
            sum[t][0] = sum[t][1] = 0.f;
        }

        // L: octets of columns in use (the others of the tile are left out)
        const auto step = [&](int i, auto edge, auto octets) {
            constexpr bool kEdge = decltype(edge)::value;
            constexpr int L = decltype(octets)::value;
            copies_wait<kStages - 2>();
            __syncwarp();
            issue();
            const unsigned char *chunk = ring + (i % kStages) * kBytes;
            const int t0 = (c0 + warp + i * kWarps) * kChunk;

            // logits: rows r8 and r8 + 8, two columns each
            float_pair x[L][2];
            {
                const uint4 ka = *reinterpret_cast<const uint4 *>(chunk + lane * 16);
                const uint4 kb = *reinterpret_cast<const uint4 *>(chunk + 512 + lane * 16);
                float s0[NG], s1[NG];
                load_halves<NG>(chunk + 2 * kCodeBytes + r8 * 2 * NG, s0);
                load_halves<NG>(chunk + 2 * kCodeBytes + (r8 + 8) * 2 * NG, s1);
                uint32_t m0 = 0, m1 = 0;
                if (j4 < NG) {
                    const uint16_t *m = reinterpret_cast<const uint16_t *>(chunk + 2 * kCodeBytes + 32 * NG);
                    m0 = m[r8 * NG + j4] * 0x10001u;
                    m1 = m[(r8 + 8) * NG + j4] * 0x10001u;
                }
#pragma unroll
                for (int t = 0; t < L; ++t) {
                    float c[4];
                    mma8_zero(c, m0, m1, kSharedQ ? s_sum[t][lane] : qs[kSharedQ ? 0 : t].sum);
                    x[t][0] = mul2(pair(c[0], c[1]), pair(0x1p-6f, 0x1p-6f));
                    x[t][1] = mul2(pair(c[2], c[3]), pair(0x1p-6f, 0x1p-6f));
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float acc[L][4];
#pragma unroll
                    for (int y = g * 4 / NG; y < (g + 1) * 4 / NG; ++y) {
                        uint32_t wa = y == 0 ? ka.x : y == 1 ? ka.y : y == 2 ? ka.z : ka.w;
                        uint32_t wb = y == 0 ? kb.x : y == 1 ? kb.y : y == 2 ? kb.z : kb.w;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
#pragma unroll
                            for (int t = 0; t < L; ++t) {
                                const uint2 f = kSharedQ ? s_frag[t][y][u][lane] : qs[kSharedQ ? 0 : t].f[y][u];
                                if (y == g * 4 / NG && u == 0)
                                    mma16_zero(acc[t], wa & 0x000f000fu, wb & 0x000f000fu, wa & 0x00f000f0u,
                                               wb & 0x00f000f0u, f.x, f.y);
                                else
                                    mma16(acc[t], wa & 0x000f000fu, wb & 0x000f000fu, wa & 0x00f000f0u,
                                          wb & 0x00f000f0u, f.x, f.y);
                            }
                            wa >>= 8;
                            wb >>= 8;
                        }
                    }
#pragma unroll
                    for (int t = 0; t < L; ++t) {
                        x[t][0] = fma2(pair(s0[g], s0[g]), pair(acc[t][0], acc[t][1]), x[t][0]);
                        x[t][1] = fma2(pair(s1[g], s1[g]), pair(acc[t][2], acc[t][3]), x[t][1]);
                    }
                }
            }

            // V steps and minima: tokens 2 j4, 2 j4 + 1 and the same 8 further, of each group
            uint32_t vs[NG][2], vm[2] = {0, 0}, any_step = 0;
            const unsigned char *v_meta = chunk + 2 * kCodeBytes + 64 * NG + j4 * 8 * NG;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (NG >= 2 && g % 2 == 0) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(v_meta + 8 * g);
                    vs[g][0] = w.x, vs[g][1] = w.y, vs[(g + 1) % NG][0] = w.z, vs[(g + 1) % NG][1] = w.w;
                } else if (NG == 1) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(v_meta);
                    vs[g][0] = w.x, vs[g][1] = w.y;
                }
            }
            if (r8 < NG) {
                const uint2 w = *reinterpret_cast<const uint2 *>(v_meta + 32 * NG + 8 * r8);
                vm[0] = w.x;
                vm[1] = w.y;
            }
            if (kEdge && t0 + kChunk > q.len) {   // behind the last token anything may lie
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int tok = t0 + 8 * h + 2 * j4;
                    const uint32_t keep = (tok < q.len ? 0xffffu : 0u) | (tok + 1 < q.len ? 0xffff0000u : 0u);
                    vm[h] &= keep;
#pragma unroll
                    for (int g = 0; g < NG; ++g) vs[g][h] &= keep;
                }
            }
            if (kEdge) {
                // A weight of zero does not keep a NaN out of a product, so what is not finite (all
                // ones in an fp16's exponent: the top bit of each half) leaves the operands here, and
                // the columns that attend such a token get their NaN in its group's minima.
                const auto not_finite = [](uint32_t w) { return ((w & 0x7fff7fffu) + 0x04000400u) & 0x80008000u; };
                const auto halves = [](uint32_t top_bits) { return (top_bits >> 15) * 0xffffu; };
                uint32_t lost = not_finite(vm[0]) | not_finite(vm[1]);
#pragma unroll
                for (int g = 0; g < NG; ++g) lost |= not_finite(vs[g][0]) | not_finite(vs[g][1]);
                if (__any_sync(~0u, lost)) {
                    int first = INT_MAX;          // such token of group r8
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int tok = t0 + 8 * h + 2 * j4;
                        lost = not_finite(vm[h]);
                        vm[h] &= ~halves(lost);
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const uint32_t x = not_finite(vs[g][h]);
                            vs[g][h] &= ~halves(x);
                            if (g == r8) lost |= x;
                        }
                        if (lost >> 31) first = min(first, tok + 1);
                        if (lost & 0x8000u) first = min(first, tok);
                    }
                    first = min(first, __shfl_xor_sync(~0u, first, 1));
                    first = min(first, __shfl_xor_sync(~0u, first, 2));
                    if (r8 < NG) {
#pragma unroll
                        for (int t = 0; t < L; ++t)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                if (first < keys_of(t, c)) z[t][c] = __int_as_float(0x7fffffff);
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                vs[g][0] = mul_half2(vs[g][0], up[g]);
                vs[g][1] = mul_half2(vs[g][1], up[g]);
                any_step |= vs[g][0] | vs[g][1];
            }

            // weights
            float y[L][4], top = -INFINITY;
#pragma unroll
            for (int t = 0; t < L; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 v = unpair(fma2(x[t][h], pair(factor[t][0], factor[t][1]), pair(-base[t][0], -base[t][1])));
                    y[t][2 * h] = v.x;
                    y[t][2 * h + 1] = v.y;
                }
            if (kEdge) {
#pragma unroll
                for (int t = 0; t < L; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (t0 + r8 + 4 * (e & 2) >= keys_of(t, e & 1)) y[t][e] = -INFINITY;
            }
#pragma unroll
            for (int t = 0; t < L; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, y[t][e]);
            // a maximum to follow, or scaled steps of 2 and more (bit 14 of an fp16 that is >= 0)
            if (__any_sync(~0u, top > kTop + kSlack || (any_step & 0x40004000u))) {
                if (__any_sync(~0u, any_step & 0x40004000u)) {
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        uint32_t raw[2], most = 0;                    // the steps themselves, 0 where masked
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t used = (vs[g][h] & 0x7fffu ? 0xffffu : 0u) | (vs[g][h] & 0x7fff0000u ? 0xffff0000u : 0u);
                            raw[h] = shared_word(smem_addr(v_meta) + 8 * g + 4 * h) & used;
                            most = max(most, max(raw[h] & 0x7fffu, raw[h] >> 16 & 0x7fffu));
                        }
                        const int e = (int)(__reduce_max_sync(~0u, most) >> 10) - 15;    // of the largest
                        const int old = exponent_of(up[g]);
                        if (e + old >= 1) {
                            const int now = e >= 1 ? -e : -2 - e;
                            const float less = pow2f(now - old);
                            up[g] = power_pair(now);
#pragma unroll
                            for (int h = 0; h < 2; ++h) vs[g][h] = mul_half2(raw[h], up[g]);
#pragma unroll
                            for (int t = 0; t < L; ++t)
#pragma unroll
                                for (int m = 2 * (g * 4 / NG); m < 2 * ((g + 1) * 4 / NG); ++m)
#pragma unroll
                                    for (int x = 0; x < 4; ++x) o[t][m][x] *= less;
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < L; ++t)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const bool out0 = y[t][c] == -INFINITY, out1 = y[t][c + 2] == -INFINITY;
                        const float2 x0 = unpair(x[t][0]), x1 = unpair(x[t][1]);
                        const float l0 = out0 ? -INFINITY : (c ? x0.y : x0.x) * factor[t][c];
                        const float l1 = out1 ? -INFINITY : (c ? x1.y : x1.x) * factor[t][c];
                        float m = fmaxf(l0, l1);
#pragma unroll
                        for (int d = 4; d < 32; d *= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
                        const float old = base[t][c], b = fmaxf(old, m - kTop);
                        const float keep = b == -INFINITY ? 1.f : exp2f(old - b);
                        base[t][c] = b;
                        sum[t][c] *= keep;
                        z[t][c] *= keep;
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            o[t][d][c] *= keep;
                            o[t][d][c + 2] *= keep;
                        }
                        y[t][c] = out0 ? -INFINITY : l0 - b;
                        y[t][c + 2] = out1 ? -INFINITY : l1 - b;
                    }
            }
            uint32_t p[L][2];
#pragma unroll
            for (int t = 0; t < L; ++t) {
#pragma unroll
                for (int e = 0; e < 4; ++e) y[t][e] = fast_exp2(y[t][e]);
                const float2 v = unpair(add2(pair(sum[t][0], sum[t][1]), add2(pair(y[t][0], y[t][1]), pair(y[t][2], y[t][3]))));
                sum[t][0] = v.x;
                sum[t][1] = v.y;
                p[t][0] = transpose8(pack_half2(y[t][0], y[t][1]));
                p[t][1] = transpose8(pack_half2(y[t][2], y[t][3]));
                float low[4];
                mma16_zero(low, vm[0], 0, vm[1], 0, p[t][0], p[t][1]);
                add_to(z[t][0], z[t][1], low[0], low[1]);
            }

            // values
            const uint4 va = *reinterpret_cast<const uint4 *>(chunk + kCodeBytes + lane * 16);
            const uint4 vb = *reinterpret_cast<const uint4 *>(chunk + kCodeBytes + 512 + lane * 16);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t ps[L][2];
#pragma unroll
                for (int t = 0; t < L; ++t) {
                    ps[t][0] = mul_half2(p[t][0], vs[g][0]);
                    ps[t][1] = mul_half2(p[t][1], vs[g][1]);
                }
#pragma unroll
                for (int m = g * 4 / NG; m < (g + 1) * 4 / NG; ++m) {
                    const uint32_t sel = m & 1 ? 0x7632 : 0x5410;
                    uint32_t wa = __byte_perm(m < 2 ? va.x : va.y, m < 2 ? va.z : va.w, sel);
                    uint32_t wb = __byte_perm(m < 2 ? vb.x : vb.y, m < 2 ? vb.z : vb.w, sel);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
#pragma unroll
                        for (int t = 0; t < L; ++t) {
                            float v[4], *sums = o[t][2 * m + u];
                            mma16_zero(v, wa & 0x000f000fu, wa & 0x00f000f0u, wb & 0x000f000fu, wb & 0x00f000f0u, ps[t][0],
                                       ps[t][1]);
                            add_to(sums[0], sums[1], v[0], v[1]);
                            add_to(sums[2], sums[3], v[2], v[3]);
                        }
                        wa >>= 8;
                        wb >>= 8;
                    }
                }
            }
        };
        // chunks that every column sees whole, then those at the causal edge or the end
        const int whole = min_keys / kChunk - c0 > warp ? (min_keys / kChunk - c0 - warp + kWarps - 1) / kWarps : 0;
        const auto walk = [&](auto octets) {
            int i = 0;
            for (; i < min(whole, mine); ++i) step(i, std::false_type(), octets);
            for (; i < mine; ++i) step(i, std::true_type(), octets);
        };
        if (NT == 1 || octets == 1)
            walk(std::integral_constant<int, 1>());
        else if (NT == 2 || octets == 2)
            walk(std::integral_constant<int, NT < 2 ? NT : 2>());
        else if (octets == 3)
            walk(std::integral_constant<int, NT < 3 ? NT : 3>());
        else
            walk(std::integral_constant<int, NT>());
        copies_wait<0>();
        __syncwarp();

        // -- join the warps -----------------------------------------------------------
        float *mine_o = reinterpret_cast<float *>(ring);             // [kCols][kOutStride]
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = sum[t][c];
#pragma unroll
                for (int d = 4; d < 32; d *= 2) l += __shfl_xor_sync(~0u, l, d);
                const int col = t * 8 + 2 * j4 + c;
                if (r8 == 0) ml[warp][col] = make_float2(base[t][c], l);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float low_part = __shfl_sync(~0u, z[t][c], (m * NG / 4) * 4 + j4);
                    float4 v;
                    const float high = pow2f(24 - exponent_of(up[m * NG / 4])), low = high * 0x1p-4f;
                    v.x = fmaf(o[t][2 * m][c], high, low_part);
                    v.y = fmaf(o[t][2 * m][c + 2], low, low_part);
                    v.z = fmaf(o[t][2 * m + 1][c], high, low_part);
                    v.w = fmaf(o[t][2 * m + 1][c + 2], low, low_part);
                    *reinterpret_cast<float4 *>(mine_o + col * kOutStride + 32 * m + 4 * r8) = v;
                }
            }
        }
        __syncthreads();
        const bool opens = c0 == 0, closes = c1 == chunks;
        for (int col = warp; col < kCols; col += kWarps) {
            const int cc = tile * kCols + col, i = cc / a.g, head = kv * a.g + cc % a.g, row = q.row0 + i;
            if (i >= q.rows) continue;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][col].x);
            float l = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 e = ml[w][col];
                const float f = e.x == -INFINITY ? 0.f : exp2f(e.x - top);
                const float4 x = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem + w * kRing) +
                                                                   col * kOutStride + 4 * lane);
                l += e.x == -INFINITY ? e.y : f * e.y;       // a NaN's sum stays one
                v.x = fmaf(f, x.x, v.x);
                v.y = fmaf(f, x.y, v.y);
                v.z = fmaf(f, x.z, v.z);
                v.w = fmaf(f, x.w, v.w);
            }
            if (opens && closes) {
                store_row(a, row, head, lane, v, top, l);
            } else {
                const long long slot = ((long long)blockIdx.x * 2 + (opens ? 1 : 0)) * kCols + col;
                *reinterpret_cast<float4 *>(sc.o + slot * kHeadDim + 4 * lane) = v;
                if (lane == 0) sc.ml[slot] = make_float2(top, l);
            }
        }
        if (opens && !closes && tid == 0) {
            const long long last = next - 1;                 // and the block that has it
            const long long ends = longer * (share + 1);       // of the longer blocks
            const int b = (int)(last < ends ? quotient(last, share + 1) : longer + quotient(last - ends, share));
            sc.open[blockIdx.x] = Open{b - (int)blockIdx.x + 1, q.row0, q.rows, kv, tile};
        }
        __syncthreads();
        at = item0 = next;
        ++tile;
    }
}

// Joins the parts of the items that several blocks share: part 0 in the first
// block's second slot, the others in the first slots of the blocks behind it.
// A task is a column of an open item.  With 8 parts and more to an item a block
// takes a task, its warps a share of the parts each; else a warp does.
constexpr int kJoinWarps = 8;

template <int NT>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(QAttn a, Scratch sc, int blocks) {
    constexpr int kCols = 8 * NT;
    constexpr int kMost = kSm * blocks_per_sm<1>(), kEach = (kMost + kJoinWarps * 32 - 1) / (kJoinWarps * 32);
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

// Columns of a tile.  Where every request has max_q rows, as many as it has, up to 32.
// Where the rows differ, what most of them fill, by the mean that the host knows: 32
// requests up to 8192 of 4 heads a kv head, with 1 to n tokens each, take with tiles of 8, 16
// and 32 columns 38, 42, 50 us (n = 2), 45, 47, 54 (3), 52, 50, 59 (4), 78, 67, 76 (8),
// 125, 103, 107 (16); all with 6 tokens 86 with 16 and 73 with 32, with 8 97 and 94.  64 up to
// 4096, most of which have one token: 63 and one of 128 92, 87, 98 us, 60 and four of 64
// 118, 107, 115, 56 and eight of 16 75, 73, 84, one token each 42, 46, 55.
int tile_columns(const QAttn &a) {
    const long long cols = (long long)a.max_q * a.g, all = (long long)a.total_q * a.g;
    const bool ragged = a.cu && a.total_q != (long long)a.batch * a.max_q;
    if (cols <= 8 || (ragged && all <= 8ll * a.batch)) return 8;
    return cols <= 16 || (ragged && all <= 32ll * a.batch) ? 16 : 32;
}

int blocks_of(const QAttn &a) {
    const int cols = tile_columns(a);
    const int per_sm = cols == 8 ? blocks_per_sm<1>() : cols == 16 ? blocks_per_sm<2>() : blocks_per_sm<4>();
    // no more than the longest lengths that the table can hold would use
    const long long rows = a.cu ? a.total_q : (long long)a.batch * a.max_q;
    const double items = (double)a.c.h_kv * (rows * a.g / cols + a.batch);
    if (a.whole) return items < (double)kSm * per_sm ? (int)items : kSm * per_sm;
    const double chunks = items * ((double)a.max_pages * (a.c.page_size / kChunk) + item_chunks<4>());
    const int most = kSm * per_sm;
    return chunks < (double)most * kMinChunks ? (int)(chunks / kMinChunks) + 1 : most;
}

// Short caches are not worth cutting: an item stays with one block, and the second launch
// falls away.
bool whole_items(const QAttn &a) { return (long long)a.max_pages * (a.c.page_size / kChunk) <= kWholeChunks; }

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <int NG, int NT>
cudaError_t launch(const QAttn &a, const Scratch &sc, int blocks, cudaStream_t st) {
    constexpr int smem = kWarps * stages<NT>() * (2 * kCodeBytes + 128 * NG);
    static_assert(stages<NT>() * (2 * kCodeBytes + 128 * NG) >= 8 * NT * kOutStride * 4, "a warp's result fits its ring");
    cudaError_t e = cudaSuccess;
    if (smem > 46 * 1024)       // above the default limit, with the static part
        e = cudaFuncSetAttribute(attn_kernel<NG, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if ((e = launch_chained(attn_kernel<NG, NT>, blocks, kThreads, smem, st, a, sc)) != cudaSuccess) return e;
    if (a.whole) return cudaSuccess;
    return launch_chained(join_kernel<NT>, blocks < 2 * kSm ? blocks : 2 * kSm, kJoinWarps * 32, 0, st, a, sc, blocks);
}

template <int NT>
cudaError_t launch_groups(const QAttn &a, const Scratch &sc, int blocks, cudaStream_t st) {
    switch (a.c.groups) {
        case 4: return launch<4, NT>(a, sc, blocks, st);
        case 2: return launch<2, NT>(a, sc, blocks, st);
        default: return launch<1, NT>(a, sc, blocks, st);
    }
}

}  // namespace

size_t qcache_attn_scratch_bytes(const QAttn &args) {
    QAttn a = args;
    a.whole = whole_items(a);
    const size_t n = blocks_of(a), cols = tile_columns(a);
    return align256(n * sizeof(Open)) + align256(n * 2 * cols * sizeof(float2)) + n * 2 * cols * kHeadDim * sizeof(float);
}

cudaError_t launch_qcache_attn(const QAttn &args, void *scratch, cudaStream_t st) {
    QAttn a = args;
    a.whole = whole_items(a);
    const size_t n = blocks_of(a), cols = tile_columns(a);
    char *p = static_cast<char *>(scratch);
    Scratch sc;
    sc.open = reinterpret_cast<Open *>(p);
    p += align256(n * sizeof(Open));
    sc.ml = reinterpret_cast<float2 *>(p);
    p += align256(n * 2 * cols * sizeof(float2));
    sc.o = reinterpret_cast<float *>(p);
    switch (cols) {
        case 8: return launch_groups<1>(a, sc, (int)n, st);
        case 16: return launch_groups<2>(a, sc, (int)n, st);
        default: return launch_groups<4>(a, sc, (int)n, st);
    }
}

}  // namespace fp
