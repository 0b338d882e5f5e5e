// fp_rope and fp_cache_append: rotary positions, on rows and on the way into a
// bf16 or e4m3 paged cache.
//
// A pair (a, b) of dims of a token at position p turns by p * f radians.  The frequency is
// held as the 64-bit fixed-point fraction of a turn that one position makes, so that p times
// it, modulo 2^64, is the angle modulo whole turns exactly: its upper 32 bits are
// the angle to 2^-32 of a turn at any position, where an fp32 product would be off by a
// radian at position 2^24, and the way there is integer arithmetic of full rate.  As an fp32,
// for sincospif, it is rounded by up to 2^-26 of a turn: 2^-23 radians, beside bf16's 2^-8.
//
// A warp takes a token (or a share of its heads, where there are few tokens): it computes
// the token's 64 cosines and sines once, and its four groups of 8 lanes then take a head's
// row each, 2 x 16 bytes a lane: the 8 first and the 8 second elements of 8 pairs (half
// layout), or 4 pairs in each (interleaved).  A rotation touches nothing but its own
// lane's elements, so rows may be rotated in place.
//
// A row of a page is one run of h_kv * 128 elements, as is a page, so a slot is a row.
//
// Bounds: memory.  65536 tokens of 32 heads (1.07 GB) 175 us, 6.1 TB/s, 0.90 of the measured
// copy rate; their projections into bf16 pages (32/4 heads, 1.34 GB) 218 us, 0.91.  At 80
// registers 24 warps an SM hold 2 rows a group in flight; with 3 rows ahead (94 registers, 16
// warps) it took 203, with 64 registers (spills) 243, with 1 row ahead 195.  e4m3
// outputs: 176 us (floor 119), 254 us into pages of 8 heads (179); two thirds of the issue slots and
// half of DRAM's rate, so instructions and the loads' latency between them, at 22 warps an SM.
// Below some thousand tokens a launch and one chain: 2.7 us.
#include "cache.cuh"

namespace fp {
namespace {

constexpr int kWarps = 8;
constexpr int kAhead = 2;                      // rows of a group whose loads are in flight together
constexpr int kSm = 152;

enum Layout { kHalf, kInterleaved, kScalar };  // kScalar: half layout, rot / 2 not a multiple of 8

struct Row {
    const __nv_bfloat16 *in;
    long long out;                             // first element
    int part, head;                            // part 0: q, 1: k, 2: v; -1: nothing to do
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t e4m3_four(const float *x, float inv) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}
__device__ __forceinline__ void unpack8(uint4 w, float *x) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(v[e] << 16);
        x[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(void *out, long long at, const float *x, bool fp8, float inv) {
    if (fp8)
        *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(out) + at) =
            make_uint2(e4m3_four(x, inv), e4m3_four(x + 4, inv));
    else
        __stcs(reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + at),
            make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7])));
}

template <Layout L>
__global__ void __launch_bounds__(kWarps * 32) rotate_kernel(RotateRows r, int shares) {
    __shared__ __align__(16) float s_cos[kWarps][64], s_sin[kWarps][64];
    // kScalar: rows in shared memory (with 2-byte loads of global memory 20000 tokens of 8 heads, 100
    // dims of 128 turned, took 82 us instead of 44)
    __shared__ __align__(16) __nv_bfloat16 s_row[L == kScalar ? kWarps * 4 : 1][kAhead][kHeadDim];
    after_previous();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, group = lane >> 3, l = lane & 7;
    const long long job = (long long)blockIdx.x * kWarps + warp;
    const int token = (int)(job / shares), share = (int)(job - (long long)token * shares);
    if (token >= r.rows) return;
    const int half = r.positions ? r.rot.rot / 2 : 0;
    if (half) {
        const long long p = r.positions[token];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int pair = lane + 32 * i;
            float s = 0.f, c = 0.f;
            if (pair < half) {
                const unsigned long long t = (unsigned long long)p * r.rot.turns[pair];
                sincospif((float)(int)(uint32_t)(t >> 32) * 0x1p-31f, &s, &c);
            }
            s_cos[warp][pair] = c * r.rot.scale;
            s_sin[warp][pair] = s * r.rot.sin_scale;
        }
        __syncwarp();
    }
    // pairs of this lane: 8 l .. 8 l + 7, or 4 l .. and 32 + 4 l ..
    float c[8], s[8];
    bool turns[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int pair = L == kInterleaved ? 4 * l + (e & 3) + 8 * (e & 4) : 8 * l + e;
        turns[e] = pair < half;
        c[e] = half ? s_cos[warp][pair] : 0.f;
        s[e] = half ? s_sin[warp][pair] : 0.f;
    }
    // first and second element of pair 8 l + e, and where the lane's two runs of 8 start
    const auto first = [&](int pair) { return pair < half ? pair : half + 2 * (pair - half) + half; };
    const auto second = [&](int pair) { return pair < half ? pair + half : half + 2 * (pair - half) + 1 + half; };
    const int run0 = L == kInterleaved ? 8 * l : L == kHalf && half > 8 * l ? 8 * l : 16 * l;
    const int run1 = L == kInterleaved ? 8 * l + 64 : L == kHalf && half > 8 * l ? 8 * l + half : 16 * l + 8;

    long long slot = -1;
    if (r.slots) {
        slot = r.slots[token];
        if (slot < -1 || slot >= r.num_slots) {
            if (lane == 0 && share == 0) set_status(r.status, FP_ERR_DEVICE_BOUNDS);
            slot = -1;
        }
    }
    const int all = r.q.heads + r.k.heads + r.v.heads;
    const int from = (int)((long long)all * share / shares), to = (int)((long long)all * (share + 1) / shares);
    const auto row_of = [&](int h) {
        Row row;
        row.part = h < r.q.heads ? 0 : h < r.q.heads + r.k.heads ? 1 : 2;
        const RowsPart &p = row.part == 0 ? r.q : row.part == 1 ? r.k : r.v;
        row.head = h - (row.part == 0 ? 0 : row.part == 1 ? r.q.heads : r.q.heads + r.k.heads);
        row.in = p.in + token * p.in_tok + row.head * p.in_head;
        row.out = (row.part == 0 ? (long long)token : slot) * p.out_tok + row.head * p.out_head;
        if (h >= to || (row.part && slot < 0)) row.part = -1;
        return row;
    };
    for (int h0 = from; h0 < to; h0 += 4 * kAhead) {
        Row row[kAhead];
        uint4 w[kAhead][2];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            row[i] = row_of(h0 + 4 * i + group);
            if (row[i].part < 0) continue;
            w[i][0] = __ldcs(reinterpret_cast<const uint4 *>(row[i].in + run0));
            w[i][1] = __ldcs(reinterpret_cast<const uint4 *>(row[i].in + run1));
        }
        // pairs that lie across the runs of 8 meet through shared memory
        __nv_bfloat16 (*mine)[kHeadDim] = s_row[L == kScalar ? warp * 4 + group : 0];
        if (L == kScalar) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (row[i].part < 0) continue;
                *reinterpret_cast<uint4 *>(mine[i] + run0) = w[i][0];
                *reinterpret_cast<uint4 *>(mine[i] + run1) = w[i][1];
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const RowsPart &p = row[i].part == 0 ? r.q : row[i].part == 1 ? r.k : r.v;
            const bool live = row[i].part >= 0, fp8 = p.scale != nullptr;
            if (L != kScalar && !live) continue;
            float x[8], y[8];
            if (L == kScalar) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = __bfloat162float(mine[i][first(8 * l + e)]);
                    y[e] = __bfloat162float(mine[i][second(8 * l + e)]);
                }
            } else {
                unpack8(w[i][0], x);
                unpack8(w[i][1], y);
            }
            if (row[i].part < 2) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float &a = L != kInterleaved ? x[e] : e < 4 ? x[2 * e] : y[2 * e - 8];
                    float &b = L != kInterleaved ? y[e] : e < 4 ? x[2 * e + 1] : y[2 * e - 7];
                    const float u = fmaf(a, c[e], -(b * s[e])), v = fmaf(b, c[e], a * s[e]);
                    if (turns[e]) {
                        a = u;
                        b = v;
                    }
                }
            }
            const float inv = live && fp8 ? 1.f / p.scale[row[i].head] : 1.f;
            if (L != kScalar) {
                store8(p.out, row[i].out + run0, x, fp8, inv);
                store8(p.out, row[i].out + run1, y, fp8, inv);
            } else {
                __syncwarp();                    // the row is read: its results take its place
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int a = first(8 * l + e), b = second(8 * l + e);
                    if (fp8) {
                        const __nv_fp8x2_storage_t z =
                            __nv_cvt_float2_to_fp8x2(make_float2(x[e] * inv, y[e] * inv), __NV_SATFINITE, __NV_E4M3);
                        reinterpret_cast<unsigned char *>(mine[i])[a] = (unsigned char)(z & 0xff);
                        reinterpret_cast<unsigned char *>(mine[i])[b] = (unsigned char)(z >> 8);
                    } else {
                        mine[i][a] = __float2bfloat16_rn(x[e]);
                        mine[i][b] = __float2bfloat16_rn(y[e]);
                    }
                }
                __syncwarp();
                const uint4 *from = reinterpret_cast<const uint4 *>(mine[i]);
                if (live && fp8) {
                    *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(p.out) + row[i].out + 16 * l) = from[l];
                } else if (live) {
                    uint4 *to = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + row[i].out) + 2 * l;
                    to[0] = from[2 * l];
                    to[1] = from[2 * l + 1];
                }
            }
        }
        if (L == kScalar) __syncwarp();
    }
}

}  // namespace

cudaError_t launch_rotate_rows(const RotateRows &r, cudaStream_t st) {
    const int all = r.q.heads + r.k.heads + r.v.heads;
    // few tokens: a warp for every four rows of a token, down to as many as fill the SMs twice
    const long long want = (16ll * kSm + r.rows - 1) / r.rows, most = (all + 3) / 4;
    const int shares = (int)(want < 1 ? 1 : want < most ? want : most);
    const long long blocks = ((long long)r.rows * shares + kWarps - 1) / kWarps;
    const bool vector = !r.positions || (r.rot.rot / 2) % 8 == 0;
    const auto kernel = r.positions && r.rot.interleaved ? rotate_kernel<kInterleaved>
                        : vector                         ? rotate_kernel<kHalf>
                                                         : rotate_kernel<kScalar>;
    return launch_chained(kernel, (unsigned)blocks, kWarps * 32, 0, st, r, shares);
}

}  // namespace fp
