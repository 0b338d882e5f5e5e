// fp_cache_attn for requests of many rows: tiles of 256 (query, head) rows on tcgen05.
//
// A kv head's rows of a request -- query by query, the g heads of a query together -- are cut
// into tiles of 2 x 128; every 128 keys and values are loaded once for both halves:
//   S_t = Q_t K^T,   O_t += P_t V,   t = 0, 1,
// with S, P (over S, as packed 16-bit pairs) and O in TMEM (2 x (128 + 128) of its 512
// columns).  The halves alternate, so that one half's softmax runs beside the other's products.
// A bf16 cache takes bf16 operands (e4m3 queries exactly, weights rounded to bf16).  Of an
// e4m3 one keys are taken as they are, against e4m3 queries, or two e4m3 terms of bf16 ones;
// values become fp16, exactly, on their way through shared memory, against weights in fp16.
// Weights are 2^(logit - m + 10), m following when the logits pass it by 4; sums, maxima and
// outputs are fp32.
//
// Work: the (request, kv head, tile) items laid end to end, each as long as its start and end
// cost plus the keys that its rows attend, are cut into equal ranges, one for each SM: the
// lengths are the GPU's, the triangle below a prompt's diagonal is weighed in, and few rows
// over a long cache spread over all SMs.  Lengths are counted in keys times g, which makes a
// tile's weight linear in its number, and sums and searches closed.  An item that a range's
// end cuts leaves partial results to the join.
//
// Roles (16 warps): the issuer of products, the walk over the items, queries (a warp a half,
// which brings the next item's while this one ends), loaders, and a softmax warpgroup for each
// half, a thread a row.  Tiles come by TMA through the block table: K into a ring of 2 (bf16)
// or 4, V into a ring of 2, of e4m3 through two staging tiles that the loaders convert from.
// Every wait is bounded.
//
// What a row does not attend may be anything, and a weight of zero does not keep a NaN out of
// a product: the loaders clear values behind a request's last token, and take values that are
// not finite out of the blocks that some of the tile's rows do not attend whole.  The item
// remembers from which key on a dim has one, and the rows past it get their NaN at the end.
#include <cuda.h>
#include <limits.h>

#include "cache.cuh"
#include "device_lengths.cuh"
#include "sm100.cuh"

namespace fp {
namespace {

using namespace sm100;

constexpr int kTilesThreads = 512, kTilesWarps = kTilesThreads / 32;
// Registers: 128 a thread at launch, dealt anew among the warpgroups.
constexpr int kRegsControl = 80, kRegsLoad = 80, kRegsSoftmax = 176;
static_assert(kRegsControl + kRegsLoad + 2 * kRegsSoftmax <= 4 * 128, "register split");
constexpr int kRows = 256;                       // packed rows of a tile
constexpr int kItemKeys = 384;                   // what an item's start and end cost, in keys
constexpr int kMinBlocks = 4;                    // least blocks of keys worth an SM
constexpr int kTile = kBlock * kHeadDim * 2, kHalf = kTile / 2;      // bytes; a half: 64 dims
constexpr int kSmemQ = 0, kSmemK = 2 * kTile, kSmemV = 4 * kTile, kSmemStage = 6 * kTile;

enum { QF = 0, QE = 2, KF = 4, KE = 8, VF = 12, VE = 14, SF = 16, PF = 18, OF = 20, MF = 22, ME = 24, SG = 26, SE = 28, VX = 30,
       DR = 32, kBars = 33 };
constexpr int kItemReaders = 1 + 2 + 8 + 4;      // the issuer, the queries' warps, the softmax warps, the loaders' warps

// A piece of an item, as the roles read it.
struct Item {
    int live;                                    // 0: no more
    int r, row0, lq, len, kv;
    int rows, tile;                              // packed rows of the request; tile of them
    int c0, c1;                                  // blocks of keys
    int edge;                                    // first block that not every row attends whole
    int min_keys;                                // keys of the tile's first row
    int opens, closes;
    int not_finite;                              // any of:
    int pad;
    int from[kHeadDim];                          // first key of a value that was taken out, INT_MAX: none
    signed char exponent[kRows];                 // of the power of two that a query row was multiplied by
};
struct Control {
    unsigned long long bars[kBars];
    uint32_t tmem, abort;
    long long at;
    int r, pad;
    union {
        Item item[2];
        long long sums[kTilesWarps];             // of the scan, before the roles part
    };
};
constexpr int kSmemBf16 = kSmemStage + (int)sizeof(Control) + 1024, kSmemFp8 = kSmemBf16 + kTile;
static_assert(kSmemFp8 <= 227 * 1024, "shared memory");

// The columns' sum over the whole block of threads.
__device__ __forceinline__ long long scan_all(long long n, long long *all, long long *sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    long long x = n;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const long long y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    long long sum = 0;
    x -= n;
    for (int w = 0; w < kTilesWarps; ++w) {
        const long long v = sums[w];
        if (w < warp) x += v;
        sum += v;
    }
    __syncthreads();
    *all = sum;
    return x;
}

// A request's tiles, and the units of each: base + 256 (tile + 1), keys times g.
struct Tiles {
    int n, start;
    long long base;
};
__device__ __forceinline__ Tiles tiles_in(const PAttn &a, const Request &q) {
    Tiles t;
    const long long rows = (long long)q.rows * a.g;
    t.n = rows > a.most_columns ? (int)((rows + kRows - 1) / kRows) : 0;
    t.start = q.len - q.lq;
    // a start past 2^27 counts as that: sums of weights stay in 64 bits
    t.base = (long long)a.g * (kItemKeys + min(max(t.start, 0), 1 << 27));
    return t;
}
__device__ __forceinline__ long long units_before(const Tiles &t, long long tile) {
    return tile * t.base + 128 * tile * (tile + 1);
}
__device__ __forceinline__ long long units_of(const PAttn &a, const Tiles &t) {
    const long long u = a.c.h_kv * units_before(t, t.n);
    return u < (1ll << 50) ? u : 1ll << 50;      // past any lengths that fit together
}

// What a wait needs besides its barrier.
struct Waits {
    uint32_t abort;
    int *status;
    unsigned long long limit;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
        return mbar_wait(bar, parity & 1u, abort, status, limit);
    }
};

template <bool kFp8>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if (kFp8) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t codes_to_f16(uint32_t codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3);
    return (uint32_t)h.x | (uint32_t)h.y << 16;
}
// 16-byte piece `piece` (8 dims) of row `row` of a 128 x 128 tile: two halves of 128-byte rows,
// pieces XORed by the row (the 128-byte swizzle of TMA and of the products' descriptors).
__device__ __forceinline__ uint32_t piece_at(uint32_t tile, int row, int piece) {
    return tile + (piece >> 3) * kHalf + row * 128 + (((piece ^ row) & 7) << 4);
}

// 16 bytes into shared memory, or zeros.
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// A half's 128 rows of queries into shared memory, by a warp: `mine(row)` is the address of a
// row, 0 for one that is not there.  A bf16 cache takes bf16 tiles.  An e4m3 one takes e4m3
// codes as they are; bf16 rows under a power of two, as two e4m3 terms of 4 bits each, which
// hold 8 bits exactly down to 2^-10 of the row's largest, and the rest to 2^-18 of it.
template <bool kFp8, typename F>
__device__ __forceinline__ void load_queries(const PAttn &a, const F &mine, uint32_t tile, signed char *exponent) {
    const int lane = threadIdx.x & 31;
    const bool codes = a.q_scale != nullptr;
#pragma unroll 1
    for (int set = 0; set < 4; ++set) {
        const unsigned long long own = mine(32 * set + lane);
        if (codes) {                             // 8 lanes a row, 4 rows at once
            if (kFp8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const unsigned long long p = __shfl_sync(~0u, own, 4 * i + (lane >> 3));
                    const int row = 32 * set + 4 * i + (lane >> 3), c = lane & 7;
                    copy16_or_zero(tile + row * 128 + (((c ^ row) & 7) << 4),
                                   p ? reinterpret_cast<const unsigned char *>(p) + c * 16 : static_cast<const unsigned char *>(a.q), p != 0);
                }
            } else {
                uint4 w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const unsigned long long p = __shfl_sync(~0u, own, 4 * i + (lane >> 3));
                    w[i] = p ? *reinterpret_cast<const uint4 *>(p + (lane & 7) * 16) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = 32 * set + 4 * i + (lane >> 3), c = lane & 7;
                    const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        h[e] = codes_to_f16(v[e >> 1] >> (16 * (e & 1)));
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
                        h[e] = pack16<false>(f.x, f.y);
                    }
                    st_shared_v4(piece_at(tile, row, 2 * c), make_uint4(h[0], h[1], h[2], h[3]));
                    st_shared_v4(piece_at(tile, row, 2 * c + 1), make_uint4(h[4], h[5], h[6], h[7]));
                }
            }
        } else {                                 // 16 lanes a row, 2 rows at once
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const unsigned long long p = __shfl_sync(~0u, own, 2 * i + (lane >> 4));
                const int row = 32 * set + 2 * i + (lane >> 4), c = lane & 15;
                copy16_or_zero(piece_at(tile, row, c),
                               p ? reinterpret_cast<const unsigned char *>(p) + c * 16 : static_cast<const unsigned char *>(a.q), p != 0);
            }
        }
    }
    copies_commit();
    copies_wait<0>();
    __syncwarp();
    if (kFp8 && !codes) {
        // in place: a row's 64 and 64 dims of bf16 make room for its two terms of 128 bytes
#pragma unroll 1
        for (int i0 = 0; i0 < 64; i0 += 4) {
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = ld_shared_v4(piece_at(tile, 2 * (i0 + i) + (lane >> 4), lane & 15));
            uint2 hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                float x[8], top = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[2 * e] = __uint_as_float(v[e] << 16);
                    x[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
                    top = max3f(top, fabsf(x[2 * e]), fabsf(x[2 * e + 1]));
                }
#pragma unroll
                for (int d = 1; d < 16; d *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                const int ex = fp16_scale_exp(__float_as_uint(top)) - 7;         // the largest into [2^7, 2^8)
                if ((lane & 15) == 0) exponent[2 * (i0 + i) + (lane >> 4)] = (signed char)ex;
                const float up = pow2f(ex);
                uint32_t h[4], l[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float u = x[2 * e] * up, y = x[2 * e + 1] * up;
                    h[e] = e4m3_pair(u, y);
                    const uint32_t back = codes_to_f16(h[e]);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&back));
                    l[e] = e4m3_pair(u - f.x, y - f.y);
                }
                hi[i] = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
                lo[i] = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 2 * (i0 + i) + (lane >> 4), c = lane & 15;
                const uint32_t at = tile + row * 128 + ((((c >> 1) ^ row) & 7) << 4) + (c & 1) * 8;
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(hi[i].x), "r"(hi[i].y) : "memory");
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + kHalf), "r"(lo[i].x), "r"(lo[i].y) : "memory");
            }
        }
    }
}

template <bool kFp8>
__global__ void __launch_bounds__(kTilesThreads, 1)
tiles_kernel(const PAttn a, const Scratch sc, const __grid_constant__ CUtensorMap map_k,
             const __grid_constant__ CUtensorMap map_v, unsigned long long limit_ns) {
    extern __shared__ unsigned char smem_raw[];
    // 1024-byte aligned, as the swizzle wants; addresses by offsets in the shared window
    unsigned char *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    Control &ctl = *reinterpret_cast<Control *>(smem + (kFp8 ? kSmemStage + kTile : kSmemStage));
    const uint32_t base = smem_u32(smem), bars = smem_u32(ctl.bars);
    const auto bar = [&](int k) { return bars + 8u * (uint32_t)k; };
    constexpr int kRing = kFp8 ? 4 : 2, kSlot = kTile / (kFp8 ? 2 : 1);        // tiles of K, as they come
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    after_previous();

    // -- this block's range of units ------------------------------------------------
    const int each = (a.batch + kTilesThreads - 1) / kTilesThreads;
    Request q = {0, 0, 0, 0};
    long long n = 0, total;
    for (int r = tid * each; r < min(a.batch, (tid + 1) * each); ++r) n += units_of(a, tiles_in(a, q = request_of(a, r)));
    long long low = scan_all(n, &total, ctl.sums);
    const long long want = total / ((long long)a.g * kBlock * kMinBlocks) + 1;
    const int blocks = total == 0 ? 0 : (int)(want < gridDim.x ? want : gridDim.x);
    if (tid == 0) sc.open[blockIdx.x].parts = 0;
    if ((int)blockIdx.x >= blocks) return;
    const long long share = quotient(total, blocks);
    const int longer = (int)(total - share * blocks);
    const long long first = blockIdx.x * share + min((int)blockIdx.x, longer), end = first + share + ((int)blockIdx.x < longer);
    if (low <= first && first < low + n) {
        int r = tid * each;
        if (each > 1)
            for (;; ++r) {
                n = units_of(a, tiles_in(a, request_of(a, r)));
                if (first < low + n || r + 1 == a.batch) break;
                low += n;
            }
        ctl.r = r;
        ctl.at = low;
    }
    if (tid == 0) {
        for (int k = 0; k < kBars; ++k) {
            uint32_t count = 1;
            if (k == PF || k == PF + 1 || k == SE || k == SE + 1 || k == VX || k == VX + 1) count = 128;
            if (kFp8 && (k == VF || k == VF + 1)) count = 128;
            if (k == MF || k == MF + 1 || k == QF || k == QF + 1) count = 32;
            if (k == ME || k == ME + 1) count = kItemReaders;
            mbar_init(bar(k), count);
        }
        ctl.abort = 0;
        fence_barrier_init();
        fence_proxy_async();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&ctl.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    const Waits wait = {smem_u32(&ctl.abort), a.status, limit_ns};
    // a wait of this launch or an earlier one on this status ran out: no work, so that a broken
    // launch ends in one limit and not in one for each block
    const bool dead = a.status && *reinterpret_cast<volatile int *>(a.status) == FP_ERR_TIMEOUT;

    if (warp < 4) {
        setmaxnreg_dec<kRegsControl>();
        if (dead) {
        } else if (warp == 1) {
            // ================= the walk over the items =================
            int r = ctl.r;
            q = request_of(a, r);
            Tiles t = tiles_in(a, q);
            long long item0 = ctl.at, at = first;
            int kv, tile;
            {
                const long long head = units_before(t, t.n);
                kv = min((int)quotient(first - item0, head), a.c.h_kv - 1);
                item0 += kv * head;
                int lo = 0, hi = t.n - 1;        // the last tile that starts at or before `first`
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (item0 + units_before(t, mid) <= first) lo = mid; else hi = mid - 1;
                }
                tile = lo;
                item0 += units_before(t, tile);
            }
            for (int k = 0;; ++k) {
                const int b = k & 1;
                Item &it = ctl.item[b];
                if (k >= 2) {
                    const bool got = wait(bar(ME + b), ((k >> 1) & 1) ^ 1);
                    if (!__all_sync(~0u, got)) break;
                }
                bool live = false;
                while (at < end && !live) {
                    if (tile == t.n) {
                        tile = 0;
                        ++kv;
                    }
                    while ((kv >= a.c.h_kv || t.n == 0) && r < a.batch) {     // the next request of this kernel
                        if (++r >= a.batch) break;
                        q = request_of(a, r);
                        t = tiles_in(a, q);
                        kv = tile = 0;
                    }
                    if (r >= a.batch) break;     // lengths that changed under the kernel
                    const int rows = q.rows * a.g;
                    const long long units = t.base + 256ll * (tile + 1), next = item0 + units;
                    // keys of a packed row: up to its query's own
                    const auto keys_of = [&](int row) { return max(0, min(q.len, t.start + row / a.g + 1)); };
                    const int count = max(1, (keys_of(min(kRows * (tile + 1), rows) - 1) + kBlock - 1) / kBlock);
                    const auto block_of = [&](long long unit) {
                        const long long c = (quotient(unit, a.g) - kItemKeys) / kBlock;
                        return (int)(c < 0 ? 0 : c < count ? c : count);
                    };
                    const int c0 = at <= item0 ? 0 : block_of(at - item0), c1 = end >= next ? count : block_of(end - item0);
                    if (c1 > c0) {
                        live = true;
                        if (lane == 0) {
                            it.r = r;
                            it.row0 = q.row0;
                            it.lq = q.lq;
                            it.len = q.len;
                            it.kv = kv;
                            it.rows = rows;
                            it.tile = tile;
                            it.c0 = c0;
                            it.c1 = c1;
                            it.min_keys = keys_of(kRows * tile);
                            it.edge = it.min_keys / kBlock;
                            it.opens = c0 == 0;
                            it.closes = c1 == count;
                            it.not_finite = 0;
                            if (c0 == 0 && c1 < count) {             // and the block that has its last key
                                const long long whole = (long long)a.g * (kItemKeys + (long long)kBlock * count);
                                const long long last = item0 + (whole < units ? whole : units) - 1, ends = longer * (share + 1);
                                const long long to = last < ends ? quotient(last, share + 1) : longer + quotient(last - ends, share);
                                sc.open[blockIdx.x] = Open{(int)(to < blocks ? to : blocks - 1) - (int)blockIdx.x + 1, q.row0, q.rows, kv, tile};
                            }
                        }
                        for (int d = lane; d < kHeadDim; d += 32) it.from[d] = INT_MAX;
                    }
                    at = item0 = next;
                    ++tile;
                }
                if (lane == 0) it.live = live;
                __syncwarp();
                mbar_arrive(bar(MF + b));
                if (!live) break;
            }
        } else if (warp == 0 && lane == 0) {
            // ================= the products' issuer =================
            constexpr uint32_t kIdS = kFp8 ? idesc_e4m3(128, 128, false) : idesc_bf16(128, 128, false);
            constexpr uint32_t kIdO = kFp8 ? idesc_f16(128, 128, true) : idesc_bf16(128, 128, true);
            const uint64_t dq = smem_desc_sw128(base + kSmemQ, 16, 1024), dk = smem_desc_sw128(base + kSmemK, 16, 1024);
            const uint64_t dv = smem_desc_sw128(base + kSmemV, kHalf, 1024);
            // e4m3: one term of the queries, or two
            const auto issue_s = [&](int t, int s) {
                const uint64_t qt = dq + ((t * kTile) >> 4), ks = dk + ((s * kSlot) >> 4);
                if (kFp8) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) mma_ss_f8(tmem + t * 256, qt + kk * 2, ks + kk * 2, kIdS, kk > 0);
                    if (!a.q_scale)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) mma_ss_f8(tmem + t * 256, qt + (kHalf >> 4) + kk * 2, ks + kk * 2, kIdS, true);
                } else {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                        mma_ss(tmem + t * 256, qt + off, ks + off, kIdS, kk > 0);
                    }
                }
                tc_commit(bar(SF + t));
            };
            const auto issue_o = [&](int t, int s, bool more) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ts(tmem + t * 256 + 128, tmem + t * 256 + kk * 8, dv + ((s * kTile + kk * 16 * 128) >> 4), kIdO, more || kk > 0);
            };
            uint32_t it = 0, edges = 0, phase0 = 0, phase1 = 0, items0 = 0, items1 = 0;
            for (int k = 0;; ++k) {
                const int b = k & 1;
                if (!wait(bar(MF + b), k >> 1)) break;
                const Item &item = ctl.item[b];
                const int live = item.live, count = item.c1 - item.c0, edge = kFp8 ? INT_MAX : item.edge - item.c0;
                const bool two = item.rows - item.tile * kRows > kBlock;
                mbar_arrive(bar(ME + b));
                if (!live) break;
                const auto keys_there = [&](uint32_t i) { return wait(bar(KF + i % kRing), i / kRing); };
                if (!wait(bar(QF), items0++) || (two && !wait(bar(QF + 1), items1++)) || !keys_there(it)) break;
                tc_fence_after();
                issue_s(0, it % kRing);
                if (count == 1) tc_commit(bar(QE));
                if (two) {
                    issue_s(1, it % kRing);
                    if (count == 1) tc_commit(bar(QE + 1));
                }
                tc_commit(bar(KE + it % kRing));
                // written out for both halves: as a loop over them it cost 8 %
                bool good = true;
                for (int j = 0; j < count; ++j, ++it) {
                    const uint32_t s = it & 1, s1 = (it + 1) % kRing;
                    const bool more = j + 1 < count, last = j + 2 == count;
                    good = j < edge ? wait(bar(VF + s), it >> 1) : wait(bar(VX + (edges & 1)), edges >> 1);
                    if (j >= edge) ++edges;
                    if (!good || !(good = wait(bar(PF), phase0++))) break;
                    tc_fence_after();
                    issue_o(0, s, j > 0);
                    if (more) {
                        if (!(good = keys_there(it + 1))) break;
                        tc_fence_after();
                        issue_s(0, s1);
                        if (last) tc_commit(bar(QE));
                    } else {
                        tc_commit(bar(OF));
                    }
                    if (two) {
                        if (!(good = wait(bar(PF + 1), phase1++))) break;
                        tc_fence_after();
                        issue_o(1, s, j > 0);
                    }
                    tc_commit(bar(VE + s));
                    if (more) {
                        if (two) {
                            issue_s(1, s1);
                            if (last) tc_commit(bar(QE + 1));
                        }
                        tc_commit(bar(KE + s1));
                    } else if (two) {
                        tc_commit(bar(OF + 1));
                    }
                }
                if (!good) break;
            }
            if (ld_shared_volatile(wait.abort)) {        // every product issued is done before the block leaves
                tc_commit(bar(DR));
                mbar_wait_drain(bar(DR), 0);
            }
        } else if (warp >= 2) {
            // ================= queries, a warp a half =================
            const int t = warp - 2;
            uint32_t items = 0;
            for (int k = 0;; ++k) {
                const int b = k & 1;
                if (!__all_sync(~0u, wait(bar(MF + b), k >> 1))) break;
                Item &item = ctl.item[b];
                if (!item.live) break;
                const int row0 = item.tile * kRows + t * kBlock;
                if (item.rows > row0) {
                    // the products of the item before are done with their queries
                    if (items && !__all_sync(~0u, wait(bar(QE + t), items - 1))) break;
                    const auto mine = [&](int row) -> unsigned long long {
                        const int packed = row0 + row, i = packed / a.g, head = item.kv * a.g + packed % a.g;
                        if (packed >= item.rows) return 0;
                        const long long at = (item.row0 + i) * a.q_stride_tok + head * a.q_stride_head;
                        return (unsigned long long)(static_cast<const unsigned char *>(a.q) + (a.q_scale ? at : 2 * at));
                    };
                    load_queries<kFp8>(a, mine, base + kSmemQ + t * kTile, item.exponent + t * kBlock);
                    fence_proxy_async();
                    mbar_arrive(bar(QF + t));
                    ++items;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ME + b));
            }
        }
    } else if (warp < 8) {
        setmaxnreg_dec<kRegsLoad>();
        // ================= loaders =================
        const int lw = warp - 4, lt = tid - 128;
        const int box = a.c.page_size < kBlock ? a.c.page_size : kBlock, boxes = kBlock / box;     // rows of one; boxes of a block
        const int outside = a.c.num_pages * a.c.page_size;               // reads zeros
        uint32_t nk = 0, nv = 0, nx = 0, edges = 0;      // tiles of K and V, staged ones of V, edge blocks
        for (int k = 0; !dead; ++k) {
            const int b = k & 1;
            const bool got = wait(bar(MF + b), k >> 1);
            if (!__all_sync(~0u, got)) break;
            Item &item = ctl.item[b];
            if (!item.live) break;
            const int c0 = item.c0, count = item.c1 - c0, len = item.len, kv = item.kv, edge = item.edge, min_keys = item.min_keys;
            const int *table = a.block_table + (long long)item.r * a.max_pages;
            // the row of the caches where this lane's box of a block starts
            const auto look = [&](int j) {
                const int tok = (c0 + j) * kBlock + (lane % boxes) * box;
                if (lw > 1 || j >= count || tok >= len) return outside;
                const int page = table[tok / a.c.page_size];
                if (page < 0 || page >= a.c.num_pages) {
                    set_status(a.status, FP_ERR_DEVICE_BOUNDS);
                    return outside;
                }
                return page * a.c.page_size + tok % a.c.page_size;
            };
            const auto copy = [&](const CUtensorMap *map, uint32_t dst, uint32_t full, int z) {       // a warp
                if (lane == 0) mbar_expect_tx(full, kSlot);
                __syncwarp();
                if (lane < (kFp8 ? 1 : 2) * boxes)
                    tma_load_3d(dst + (lane / boxes) * kHalf + (lane % boxes) * box * 128, map, full, (lane / boxes) * 64, kv, z);
                __syncwarp();
            };
            bool good = true;
            // K by warp 1, as far ahead as its ring goes
            const auto keys = [&](int z) {
                good = nk < kRing || __all_sync(~0u, wait(bar(KE + nk % kRing), (nk / kRing) ^ 1));
                if (good) {
                    copy(&map_k, base + kSmemK + (nk % kRing) * kSlot, bar(KF + nk % kRing), z);
                    ++nk;
                }
            };
            const auto stage = [&](int z) {              // e4m3 V, by warp 0
                good = nx < 2 || __all_sync(~0u, wait(bar(SE + (nx & 1)), (nx >> 1) ^ 1));
                if (good) {
                    copy(&map_v, base + kSmemStage + (nx & 1) * kHalf, bar(SG + (nx & 1)), z);
                    ++nx;
                }
            };
            constexpr int kAhead = kRing - 1;
            int z1 = 0;                                  // of the next tile that this warp copies
            if (lw == 1) {
                int z[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) z[i] = look(i);
                z1 = look(kAhead);
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    if (i < count && good) keys(z[i]);
            } else if (lw == 0) {
                const int z0 = look(0);
                z1 = look(1);
                if (kFp8) {
                    stage(z0);
                    if (count > 1 && good) stage(z1);
                    z1 = look(2);
                } else {
                    z1 = z0;
                }
            }
            for (int j = 0; j < count && good; ++j, ++nv) {
                const uint32_t s = nv & 1, tile = base + kSmemV + s * kTile;
                const int z = z1;
                if (lw < 2) z1 = look(j + 1 + (lw == 1 ? kAhead : kFp8 ? 2 : 0));
                if (lw == 1 && j + kAhead < count) keys(z);
                // every loader follows the ring phase by phase: a parity alone does not tell a tile from
                // the one before it
                if (!good || !(good = nv < 2 || __all_sync(~0u, wait(bar(VE + s), (nv >> 1) ^ 1)))) break;
                if (!kFp8) {
                    if (lw == 0) copy(&map_v, tile, bar(VF + s), z);
                    if (c0 + j < edge) continue;
                    // a thread a row
                    if (!(good = __all_sync(~0u, wait(bar(VF + s), nv >> 1)))) break;
                    const int key = (c0 + j) * kBlock + lt;         // can pass 2^31 behind the last token
                    if ((uint32_t)key >= (uint32_t)len) {
#pragma unroll
                        for (int p = 0; p < 16; ++p) st_shared_v4(piece_at(tile, lt, p), make_uint4(0, 0, 0, 0));
                    } else if (key >= min_keys) {
#pragma unroll 4
                        for (int p = 0; p < 16; ++p) {
                            uint4 w = ld_shared_v4(piece_at(tile, lt, p));
                            const auto bad = [](uint32_t x) { return ((x & 0x7fff7fffu) + 0x00800080u) & 0x80008000u; };
                            if (bad(w.x) | bad(w.y) | bad(w.z) | bad(w.w)) {
                                uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t x = bad(v[e]);
                                    if (x & 0x8000u) atomicMin(&item.from[8 * p + 2 * e], key);
                                    if (x >> 31) atomicMin(&item.from[8 * p + 2 * e + 1], key);
                                    v[e] &= ~((x >> 15) * 0xffffu);
                                }
                                st_shared_v4(piece_at(tile, lt, p), make_uint4(v[0], v[1], v[2], v[3]));
                                item.not_finite = 1;
                            }
                        }
                    }
                    fence_proxy_async();
                    mbar_arrive(bar(VX + (edges & 1)));
                    ++edges;
                } else {
                    if (!(good = __all_sync(~0u, wait(bar(SG + s), nv >> 1)))) break;      // the staging ring goes as V's does
                    // rows 16 p + lt / 8, dims 16 c ..  The loops stay short: what the softmax and this
                    // run at once has to fit the instruction caches
                    const uint32_t from = base + kSmemStage + s * kHalf + lt * 16;
                    const int row0 = lt >> 3, c = lt & 7, o = c >> 2;
                    const auto convert = [&](uint4 w, uint32_t (&h)[8]) {
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) h[e] = codes_to_f16(u[e >> 1] >> (16 * (e & 1)));
                    };
                    // lanes 4 .. 7 of a row write their two pieces the other way round: all banks, once
                    const auto put = [&](int row, const uint32_t (&h)[8]) {
                        const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
                        st_shared_v4(piece_at(tile, row, 2 * c + o), o ? hi : lo);
                        st_shared_v4(piece_at(tile, row, 2 * c + 1 - o), o ? lo : hi);
                    };
                    if (c0 + j < edge) {
#pragma unroll 1
                        for (int p = 0; p < 8; p += 4) {
                            uint4 w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[i] = ld_shared_v4(from + (p + i) * 2048);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t h[8];
                                convert(w[i], h);
                                put(row0 + 16 * (p + i), h);
                            }
                        }
                    } else {
#pragma unroll 1
                        for (int p = 0; p < 8; ++p) {
                            uint32_t h[8];
                            convert(ld_shared_v4(from + p * 2048), h);
                            const int key = (c0 + j) * kBlock + row0 + 16 * p;
                            const bool behind = (uint32_t)key >= (uint32_t)len;
                            uint32_t any = 0;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                if (behind) h[e] = 0;
                                any |= ((h[e] & 0x7fff7fffu) + 0x04000400u) & 0x80008000u;
                            }
                            if (any && key >= min_keys) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const uint32_t y = ((h[e] & 0x7fff7fffu) + 0x04000400u) & 0x80008000u;
                                    if (y & 0x8000u) atomicMin(&item.from[16 * c + 2 * e], key);
                                    if (y >> 31) atomicMin(&item.from[16 * c + 2 * e + 1], key);
                                    h[e] &= ~((y >> 15) * 0xffffu);
                                }
                                item.not_finite = 1;
                            }
                            put(row0 + 16 * p, h);
                        }
                    }
                    fence_proxy_async();
                    mbar_arrive(bar(VF + s));
                    // not before the codes were used: an arrival waits for no load that is on its way, and the
                    // next tile may land first
                    mbar_arrive(bar(SE + s));
                    if (lw == 0 && j + 2 < count) stage(z);
                }
            }
            if (!__all_sync(~0u, good)) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(ME + b));
        }
        // after an abort, the copies armed last land before the block leaves
        if (lw < 2 && lane == 0 && ld_shared_volatile(wait.abort)) {
            if (lw == 1) {
                for (uint32_t i = nk < kRing ? 0 : nk - kRing; i < nk; ++i) mbar_wait_drain(bar(KF + i % kRing), (i / kRing) & 1);
            } else {
                // of bf16, the one that the last wait was for may not have been armed: waiting for it runs out
                const uint32_t n = kFp8 ? nx : nv + 1;
                for (uint32_t i = n < 2 ? 0 : n - 2; i < n; ++i) mbar_wait_drain(bar((kFp8 ? SG : VF) + (i & 1)), (i >> 1) & 1);
            }
        }
    } else {
        setmaxnreg_inc<kRegsSoftmax>();
        // ================= softmax, a warpgroup a half, a thread a row =================
        const int t = (warp - 8) / 4, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t s_at = tmem + ((uint32_t)(quarter * 32) << 16) + t * 256, o_at = s_at + 128;
        uint32_t phase = 0, items = 0;
        for (int k = 0; !dead; ++k) {
            const int b = k & 1;
            const bool got = wait(bar(MF + b), k >> 1);
            if (!__all_sync(~0u, got)) break;
            const Item &item = ctl.item[b];
            if (!item.live) break;
            const int rows = item.rows, packed = item.tile * kRows + t * kBlock + row;
            if (rows - item.tile * kRows <= t * kBlock) {            // no row in this half
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ME + b));
                continue;
            }
            const bool valid = packed < rows;
            const int i = packed / a.g, head = item.kv * a.g + packed % a.g;
            const int keys = valid ? max(0, min(item.len, item.len - item.lq + i + 1)) : 0;
            float cs = a.scale * kLog2e;                             // base-2 logits
            if (kFp8) cs *= __ldg(a.k_scale + item.kv);
            if (a.q_scale && valid) cs *= __ldg(a.q_scale + head);
            const int count = item.c1 - item.c0, key0 = item.c0 * kBlock;
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int j = 0; j < count; ++j, ++phase) {
                const bool there = wait(bar(SF + t), phase);
                if (!__all_sync(~0u, there)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (kFp8 && !a.q_scale && j == 0)
                    cs *= pow2f(-*reinterpret_cast<const volatile signed char *>(&item.exponent[t * kBlock + row]));
                float x[128];
                {
                    uint32_t v[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(s_at + c * 32, v[c]);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 4; ++c) reg_fence(v[c]);
#pragma unroll
                    for (int e = 0; e < 128; ++e) x[e] = __uint_as_float(v[e >> 5][e & 31]);
                }
                const int seen = keys - key0 - j * kBlock;           // keys of this block that the row attends
                if (seen < kBlock) {
#pragma unroll
                    for (int e = 0; e < 128; ++e)
                        if (e >= seen) x[e] = -INFINITY;
                }
                float top[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) top[e] = max3f(x[3 * e], x[3 * e + 1], x[3 * e + 2]);
#pragma unroll
                for (int e = 24; e < 128; e += 2) top[(e >> 1) & 7] = max3f(top[(e >> 1) & 7], x[e], x[e + 1]);
                const float raw = fmaxf(max3f(max3f(top[0], top[1], top[2]), top[3], top[4]), max3f(top[5], top[6], top[7]));
                const float mx = raw == -INFINITY ? -INFINITY : raw * cs;
                const bool grow = mx > m + (kTop + kSlack);
                const bool any_grow = __any_sync(~0u, grow);
                float keep = 1.f;
                if (grow) {
                    keep = fast_exp2(m - (mx - kTop));               // 0 for the first
                    m = mx - kTop;
                    l *= keep;
                }
                const float off = m == -INFINITY ? 0.f : -m;
                const uint64_t cc = f2_pack(cs, cs), oo = f2_pack(off, off);
                uint64_t acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t p[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float y0, y1;
                        f2_unpack(f2_fma(f2_pack(x[64 * half + 2 * e], x[64 * half + 2 * e + 1]), cc, oo), y0, y1);
                        y0 = fast_exp2(y0);
                        y1 = fast_exp2(y1);
                        acc[e & 1] = f2_add(acc[e & 1], f2_pack(y0, y1));
                        p[e] = pack16<kFp8>(y0, y1);
                    }
                    tmem_st32(s_at + 32 * half, p);
                }
                if (any_grow && j > 0) {
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[32];
                        tmem_ld32(o_at + c * 32, o);
                        tmem_ld_wait();
                        reg_fence(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                        tmem_st32(o_at + c * 32, o);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(bar(PF + t));
                float r0, r1, r2, r3;
                f2_unpack(acc[0], r0, r1);
                f2_unpack(acc[1], r2, r3);
                l += (r0 + r1) + (r2 + r3);
            }
            if (!ok) break;
            const bool done = wait(bar(OF + t), items);
            if (!__all_sync(~0u, done)) break;
            tc_fence_after();
            const bool whole = item.opens && item.closes;
            const float v_scale = kFp8 ? __ldg(a.v_scale + item.kv) : 1.f;
            const float by = !whole ? v_scale : l == 0.f ? 0.f : v_scale / l;
            const int not_finite = *reinterpret_cast<const volatile int *>(&item.not_finite);
            const long long out_row = item.row0 + i, slot = ((long long)blockIdx.x * 2 + (item.opens ? 1 : 0)) * kRows + t * kBlock + row;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                tmem_ld32(o_at + c * 32, o);
                tmem_ld_wait();
                reg_fence(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
                if (not_finite)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (item.from[32 * c + e] < keys) o[e] = 0x7fffffffu;
                if (!valid) continue;
                if (whole) {
                    uint4 *to = reinterpret_cast<uint4 *>(a.out + (out_row * a.h_q + head) * kHeadDim + 32 * c);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        to[e] = make_uint4(pack16<false>(__uint_as_float(o[8 * e]), __uint_as_float(o[8 * e + 1])),
                                           pack16<false>(__uint_as_float(o[8 * e + 2]), __uint_as_float(o[8 * e + 3])),
                                           pack16<false>(__uint_as_float(o[8 * e + 4]), __uint_as_float(o[8 * e + 5])),
                                           pack16<false>(__uint_as_float(o[8 * e + 6]), __uint_as_float(o[8 * e + 7])));
                } else {
                    uint4 *to = reinterpret_cast<uint4 *>(sc.o + slot * kHeadDim + 32 * c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) to[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
            }
            if (valid && !whole) sc.ml[slot] = make_float2(m, l);
            else if (valid && a.lse) a.lse[(long long)head * a.total_q + out_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            // the next item's first product over O follows its weights, which follow these reads
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(ME + b));
            ++items;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode() {
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeFn)p;
    }();
    return fn;
}
// A cache as [tokens][h_kv][128]: boxes of tokens of one head, 64 dims of bf16 or 128 of e4m3,
// swizzled as the products take them or plain; a token past the last one reads zeros.
bool map_pages(CUtensorMap *m, const void *base, const Pages &c, bool fp8, bool swizzled) {
    const EncodeFn fn = encode();
    if (!fn) return false;
    const cuuint64_t esz = fp8 ? 1 : 2;
    const cuuint64_t dims[3] = {kHeadDim, (cuuint64_t)c.h_kv, (cuuint64_t)c.num_pages * c.page_size};
    const cuuint64_t strides[2] = {kHeadDim * esz, kHeadDim * esz * c.h_kv};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / esz), 1, (cuuint32_t)(c.page_size < kBlock ? c.page_size : kBlock)};
    const cuuint32_t one[3] = {1, 1, 1};
    return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides,
              box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Thread blocks: one for each SM, and no more than the longest lengths that the table holds would use.
int tiles_blocks(const PAttn &a) {
    const long long rows = a.cu ? a.total_q : (long long)a.batch * a.max_q;
    const double items = (double)a.c.h_kv * ((double)rows * a.g / kRows + a.batch);
    const double blocks = items * ((double)a.max_pages * a.c.page_size + 2 * kItemKeys) / (kBlock * kMinBlocks) + 1;
    return blocks < kSm ? (int)blocks : kSm;
}

}  // namespace

size_t cache_tiles_scratch_bytes(const PAttn &a) {
    const size_t n = tiles_blocks(a);
    return align256(n * sizeof(Open)) + align256(n * 2 * kRows * sizeof(float2)) + n * 2 * kRows * kHeadDim * sizeof(float);
}

cudaError_t launch_cache_tiles(const PAttn &a, void *scratch, unsigned long long limit_ns, cudaStream_t st) {
    const size_t n = tiles_blocks(a);
    char *p = static_cast<char *>(scratch);
    Scratch sc;
    sc.open = reinterpret_cast<Open *>(p);
    p += align256(n * sizeof(Open));
    sc.ml = reinterpret_cast<float2 *>(p);
    p += align256(n * 2 * kRows * sizeof(float2));
    sc.o = reinterpret_cast<float *>(p);
    const bool fp8 = a.k_scale != nullptr;
    CUtensorMap map_k, map_v;
    if (!map_pages(&map_k, a.c.k, a.c, fp8, true) || !map_pages(&map_v, a.c.v, a.c, fp8, !fp8)) return cudaErrorInvalidValue;
    const auto kernel = fp8 ? tiles_kernel<true> : tiles_kernel<false>;
    const int smem = fp8 ? kSmemFp8 : kSmemBf16;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if ((e = launch_chained(kernel, (unsigned)n, kTilesThreads, smem, st, a, sc, map_k, map_v, limit_ns)) != cudaSuccess) return e;
    return launch_chained(join_kernel<kRows / 8, kSm, PAttn>, (unsigned)n * 8, kJoinWarps * 32, 0, st, a, sc,
                          (int)n);
}

}  // namespace fp
