// fp_cache_attn for requests of many rows: tiles of 256 (query, head) rows on tcgen05.
//
// A kv head's rows of a request -- query by query, the g heads of a query together -- are cut
// into tiles of two halves of at most 128, whole queries each; every 128 keys and values are
// loaded once for both halves:
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
// cost plus the keys that its last row may attend, are cut into equal ranges, one for each SM:
// the lengths are the GPU's, the triangle below a prompt's diagonal is weighed in, and few rows
// over a long cache spread over all SMs.  A tile's weight is linear in its number, which makes
// sums and searches closed.  An item that a range's end cuts leaves partial results to the join.
//
// Roles (16 warps): the walk over the items, the issuer of products (and of the queries'
// copies), a thread that follows the tiles for it, the copies of keys and values (TMA, through
// the block table), loaders that convert or clean, and a softmax warpgroup for each half, a
// thread a row.  bf16 tiles of K and V share a ring of 5;
// e4m3 keys have one of 4, values one of 2 that the loaders fill from two staged tiles.  Every
// wait is bounded.  The roles' code is kept short: together it has to fit the instruction
// caches (with the conversion written out eight times a step took 5100 clocks and not 3700).
//
// Bounds: the chain from S through a half's softmax back to the next S, with the issuer's
// instructions between: 1.5 us a block of 128 keys (2900 clocks; the products alone take 2048,
// which 8 softmax warps beside them, reading and writing TMEM, do not slow).  A chunk of 2048
// behind 32785 tokens (32/4 heads, bf16, 1.13e12 FLOP) 684 to 697 us in a graph, 1630 to 1660 TFLOP/s,
// 0.84 to 0.86 of the measured burst rate (called from Python in a loop of seconds, under the power
// cap, up to 743: 0.79); e4m3 691 us with e4m3 queries, 751 with bf16 ones (two terms of S).  An
// item's start and end cost some 4 us, a launch 6 before its first block.
// What it took: the issuer not waiting for tiles itself 810 to 718, results stored by runs of
// rows 718 to 688.  Measured and left out: an issuer for each half (994 instead of 807: their
// products mix on one pipe), all lanes of the issuer's warp at its instructions (897), P handed
// over by halves (848), loops over its 8 products (832 to 1096), P packed by integers
// instead of conversions (720 instead of 685).
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
constexpr int kRows = 2 * kBlock;                // places of a tile's rows
constexpr int kItemKeys = 512;                   // what an item's start and end cost, in keys (256 to 1024: within 5 %)
constexpr int kMinBlocks = 4;                    // least blocks of keys worth an SM
// What waits that may span an item are given beside the limit, for each block of keys (and each 128 rows of
// zeros) that an item may have: 40 times what one takes.  (A count of blocks that such waits watch, so that their
// limit starts again with it, cost 3 % of a mixed step in the roles' code.)
constexpr unsigned long long kBlockNs = 64000;
constexpr int kTile = kBlock * kHeadDim * 2, kHalf = kTile / 2;      // bytes; a half: 64 dims
constexpr int kSmemQ = 0, kSmemK = 2 * kTile;
constexpr int kRingBf16 = 5;                     // K0 V0 K1 V1 ...
constexpr int kRingK = 4, kSmemV = kSmemK + kRingK * kHalf, kSmemStage = kSmemV + 2 * kTile;      // e4m3
constexpr int kSmemEnd = 7 * kTile;
static_assert(kSmemK + kRingBf16 * kTile == kSmemEnd && kSmemStage + 2 * kHalf == kSmemEnd, "shared memory");

// Barriers: queries, tiles full and empty (bf16: of the ring; e4m3: of K, then V), S ready, P
// ready, O ready, items, staged tiles (bf16: tiles to be cleaned, of which the ring may hold
// three) full and empty (cleaned).
enum { QF = 0, TF = 2, TE = 8, SF = 14, PF = 16, OF = 18, MF = 20, ME = 22, GF = 24, GE = 27, DR = 30, kBars = 31 };
constexpr int kUnclean = (kRingBf16 + 1) / 2;
static_assert(kUnclean == GE - GF, "barriers of tiles to be cleaned");
constexpr int VF = TF + kRingK, VE = TE + kRingK;
constexpr int kItemReaders = 1 + 1 + 1 + 8 + 4;  // issuer, what follows for it, copies, softmax warps, loaders' warps

// A piece of an item, as the roles read it.
struct Item {
    int live;                                    // 0: no more
    int r, row0, lq, len, kv;
    int rows, tile;                              // queries of the request; tile of them
    int c0, c1;                                  // blocks of keys (none: rows without a key)
    int edge;                                    // first block that not every row attends whole
    int min_keys;                                // keys of the tile's first row
    int opens, closes;
    int not_finite;                              // any of:
    int pad;
    int from[kHeadDim];                          // first key of a value that was taken out, INT_MAX: none
};
struct Control {
    unsigned long long bars[kBars];
    uint32_t tmem, abort;
    long long at;
    int r, dead;
    uint32_t left[4];                            // queries copied of each half, tiles of the ring, staged (or unclean) ones
    union {
        Item item[2];
        long long sums[kTilesWarps];             // of the scan, before the roles part
    };
};
constexpr int kSmem = kSmemEnd + (int)sizeof(Control) + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");

// Exclusive scan over all threads; *all is the sum.
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

// A request's tiles, and the units of each, in keys: base + queries up to its end.
struct Tiles {
    int n, start;
    long long base;
};
__device__ __forceinline__ Tiles tiles_in(const PAttn &a, const Request &q) {
    Tiles t;
    t.n = (long long)q.rows * a.g > a.most_columns ? (q.rows + 2 * a.half - 1) / (2 * a.half) : 0;
    if (q.len == 0 && t.n) t.n = 1;              // zeros for all its rows, as one item
    t.start = q.len - q.lq;
    // a start past 2^27 counts as that: sums of weights stay in 64 bits
    t.base = kItemKeys + min(max(t.start, 0), 1 << 27);
    if (q.len == 0) t.base += (long long)q.rows * a.g / 4;
    return t;
}
__device__ __forceinline__ long long units_before(const PAttn &a, const Tiles &t, long long tile) {
    return tile * t.base + a.half * tile * (tile + 1);
}
__device__ __forceinline__ long long units_of(const PAttn &a, const Tiles &t) {
    const long long u = a.c.h_kv * units_before(a, t, t.n);
    return u < (1ll << 50) ? u : 1ll << 50;      // past any lengths that fit together
}

// What a wait needs besides its barrier.  One that runs out is recorded over what was found in device data: that
// leaves results defined, and it does not; and other blocks and later launches look for it.
struct Waits {
    uint32_t abort;
    int *status;
    unsigned long long limit, item_limit;
    __device__ __forceinline__ bool bounded(uint32_t bar, uint32_t parity, unsigned long long ns) const {
        if (mbar_try_wait(bar, parity)) return true;
        const unsigned long long since = global_ns();
        for (uint32_t it = 1;; ++it) {
            if (mbar_try_wait(bar, parity)) return true;
            if ((it & 63u) == 0) {
                if (ld_shared_volatile(abort)) return false;
                if (status && *reinterpret_cast<volatile int *>(status) == FP_ERR_TIMEOUT) {
                    st_shared_volatile(abort, 1);        // another block gave up
                    return false;
                }
                if (global_ns() - since > ns) {
                    if (status) atomicExch(status, FP_ERR_TIMEOUT);
                    st_shared_volatile(abort, 1);
                    return false;
                }
            }
        }
    }
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const { return bounded(bar, parity & 1u, limit); }
    // A wait that may span an item: the walk's for the item before the last, the loaders' for an item's first edge
    // block, an idle half's for the next item.
    __device__ __forceinline__ bool through_item(uint32_t bar, uint32_t parity) const {
        return bounded(bar, parity & 1u, item_limit);
    }
};

// Products with a descriptor's low word (address and leading offset) as they come and the high
// one, alike for all 128-byte swizzled tiles here, as a constant: the issuer's time is that of
// its instructions, and half a descriptor's arithmetic is half of it.
constexpr uint32_t kDescHigh = 1024 >> 4 | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t at, uint32_t leading) { return (at >> 4 & 0x3fffu) | leading >> 4 << 16; }
__device__ __forceinline__ void product_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t more) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(more), "n"(kDescHigh)
                 : "memory");
}
__device__ __forceinline__ void product_ss_f8(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t more) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(more), "n"(kDescHigh)
                 : "memory");
}
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t more) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(more), "n"(kDescHigh)
                 : "memory");
}

// 16-byte piece `piece` (8 dims) of row `row` of a 128 x 128 tile: two halves of 128-byte rows,
// pieces XORed by the row (the 128-byte swizzle of TMA and of the products' descriptors).
__device__ __forceinline__ uint32_t piece_at(uint32_t tile, int row, int piece) {
    return tile + (piece >> 3) * kHalf + row * 128 + (((piece ^ row) & 7) << 4);
}

template <bool kFp8>
__global__ void __launch_bounds__(kTilesThreads, 1)
tiles_kernel(const PAttn a, const Scratch sc, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
             const __grid_constant__ CUtensorMap map_v, unsigned long long limit_ns, unsigned long long item_limit_ns) {
    extern __shared__ unsigned char smem_raw[];
    // 1024-byte aligned, as the swizzle wants; addresses by offsets in the shared window
    unsigned char *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    Control &ctl = *reinterpret_cast<Control *>(smem + kSmemEnd);
    const uint32_t base = smem_u32(smem), bars = smem_u32(ctl.bars);
    const auto bar = [&](int k) { return bars + 8u * (uint32_t)k; };
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    // barriers and TMEM while the kernel before ends
    if (tid == 0) {
        for (int k = 0; k < kBars; ++k) {
            uint32_t count = 1;
            if (k == PF || k == PF + 1 || (k >= GE && k < GE + kUnclean)) count = 128;
            if (kFp8 && (k == VF || k == VF + 1)) count = 128;
            if (k == PF) count = 129;
            if (k == MF || k == MF + 1) count = 32;
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
    after_previous();
    // If a wait of this launch or an earlier one on this status ran out: no work, so that a broken launch
    // ends in one limit and not in one for each block.  Read by one thread: another block may record it
    // at any time, and all lanes of a warp have to go the same way.
    const int status = tid == 0 && a.status ? *reinterpret_cast<volatile int *>(a.status) : FP_OK;

    // -- this block's range of units ------------------------------------------------
    const int each = (a.batch + kTilesThreads - 1) / kTilesThreads;
    Request q = {0, 0, 0, 0};
    long long n = 0, total;
    for (int r = tid * each; r < min(a.batch, (tid + 1) * each); ++r) n += units_of(a, tiles_in(a, q = request_of(a, r)));
    long long low = scan_all(n, &total, ctl.sums);
    const long long want = total / (kBlock * kMinBlocks) + 1;
    const int blocks = total == 0 ? 0 : (int)(want < gridDim.x ? want : gridDim.x);
    if (tid == 0) {
        sc.open[blockIdx.x].parts = 0;
        ctl.dead = status == FP_ERR_TIMEOUT;
    }
    if ((int)blockIdx.x >= blocks) {
        __syncthreads();
        if (warp == 0) tmem_dealloc(ctl.tmem, 512);
        return;
    }
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    const Waits wait = {smem_u32(&ctl.abort), a.status, limit_ns, item_limit_ns};
    const bool dead = ctl.dead;

    if (warp < 4) {
        setmaxnreg_dec<kRegsControl>();
        if (dead) {
        } else if (warp == 1) {
            // ================= the walk over the items =================
            int r = ctl.r;
            long long item0 = ctl.at, at = first;
            q = request_of(a, r);
            Tiles t = tiles_in(a, q);
            int kv, tile;
            {
                const long long head = units_before(a, t, t.n);
                kv = min((int)quotient(first - item0, head), a.c.h_kv - 1);
                item0 += kv * head;
                int lo = 0, hi = t.n - 1;        // the last tile that starts at or before `first`
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (item0 + units_before(a, t, mid) <= first) lo = mid; else hi = mid - 1;
                }
                tile = lo;
                item0 += units_before(a, t, tile);
            }
            for (int k = 0;; ++k) {
                const int b = k & 1;
                Item &it = ctl.item[b];
                if (k >= 2) {
                    const bool got = wait.through_item(bar(ME + b), ((k >> 1) & 1) ^ 1);
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
                    const long long units = t.base + 2ll * a.half * (tile + 1), next = item0 + units;
                    // keys of a query: up to its own
                    const auto keys_of = [&](int i) { return max(0, min(q.len, t.start + i + 1)); };
                    const int count = (keys_of(min(2 * a.half * (tile + 1), q.rows) - 1) + kBlock - 1) / kBlock;
                    const auto block_of = [&](long long unit) {
                        const long long c = (unit - kItemKeys) / kBlock;
                        return (int)(c < 0 ? 0 : c < count ? c : count);
                    };
                    const int c0 = at <= item0 ? 0 : block_of(at - item0), c1 = end >= next ? count : block_of(end - item0);
                    // rows without a key are the piece's that has the item's first unit
                    if (c1 > c0 || (count == 0 && at <= item0)) {
                        live = true;
                        if (lane == 0) {
                            it.r = r;
                            it.row0 = q.row0;
                            it.lq = q.lq;
                            it.len = q.len;
                            it.kv = kv;
                            it.rows = q.rows;
                            it.tile = tile;
                            it.c0 = c0;
                            it.c1 = c1;
                            it.min_keys = keys_of(2 * a.half * tile);
                            it.edge = it.min_keys / kBlock;
                            it.opens = c0 == 0;
                            it.closes = c1 == count;
                            it.not_finite = 0;
                            if (c0 == 0 && c1 < count) {             // and the block that has its last key
                                const long long whole = kItemKeys + (long long)kBlock * count;
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
            const uint32_t dq = desc_low(base + kSmemQ, 16), dk = desc_low(base + kSmemK, 16);
            const uint32_t dv = desc_low(base + (kFp8 ? kSmemV : kSmemK), kHalf);
            const int terms = kFp8 && a.q_scale ? 1 : 2;     // tiles of a half's queries: bf16 64 dims each, e4m3 a term each
            const auto issue_s = [&](int t, uint32_t slot) {
                const uint32_t qt = dq + ((t * kTile) >> 4), ks = dk + ((slot * (kFp8 ? kHalf : kTile)) >> 4);
                if (kFp8) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) product_ss_f8(tmem + t * 256, qt + kk * 2, ks + kk * 2, kIdS, kk > 0);
                    if (terms == 2)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) product_ss_f8(tmem + t * 256, qt + (kHalf >> 4) + kk * 2, ks + kk * 2, kIdS, true);
                } else {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                        product_ss(tmem + t * 256, qt + off, ks + off, kIdS, kk > 0);
                    }
                }
                tc_commit(bar(SF + t));
            };
            const auto issue_o = [&](int t, uint32_t slot, bool more) {
                const uint32_t vs = dv + ((slot * kTile) >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    product_ts(tmem + t * 256 + 128, tmem + t * 256 + kk * 8, vs + ((kk * 16 * 128) >> 4), kIdO, more || kk > 0);
            };
            // it: blocks so far.  Their tiles: bf16 K in place 2 it of the ring, V behind it
            uint32_t it = 0, phase0 = 0, phase1 = 0, items0 = 0, items1 = 0;
            for (int k = 0;; ++k) {
                const int b = k & 1;
                if (!wait(bar(MF + b), k >> 1)) break;
                const Item &item = ctl.item[b];
                if (!item.live) break;
                const int i0 = 2 * a.half * item.tile, count = item.c1 - item.c0;
                const bool two = item.rows - i0 > a.half;
                if (count) {
                    // the weights of the item before are there, so its last products with the queries are done
                    for (int t = 0; t < (two ? 2 : 1); ++t) {
                        mbar_expect_tx(bar(QF + t), terms * a.half * a.g * 128);
                        for (int x = 0; x < terms; ++x)
                            tma_load_3d(base + kSmemQ + t * kTile + x * kHalf, &map_q, bar(QF + t), kFp8 ? 0 : 64 * x, item.kv * a.g,
                                        item.row0 + i0 + t * a.half + (kFp8 ? x * a.total_q : 0));
                    }
                }
                mbar_arrive(bar(ME + b));
                if (count == 0) continue;
                ++items0;
                items1 += two;
                if (!wait(bar(QF), items0 - 1) || (two && !wait(bar(QF + 1), items1 - 1))) break;
                if (!(kFp8 ? wait(bar(TF + it % kRingK), it / kRingK) : wait(bar(TF + 2 * it % kRingBf16), 2 * it / kRingBf16))) break;
                bool good = true;
                // S of block j behind O of block j - 1, half by half; written out for both halves (as a
                // loop over them it cost 8 %)
                for (int j = 0; j <= count; ++j) {
                    const uint32_t vs = kFp8 ? (it - 1) & 1 : (2 * it - 1) % kRingBf16, ks = kFp8 ? it % kRingK : (2 * it) % kRingBf16;
                    if (j > 0) {
                        // the first half's weights, V of this block and K of the next
                        if (!(good = wait(bar(PF), phase0++))) break;
                        tc_fence_after();
                        issue_o(0, vs, j > 1);
                        if (j == count) tc_commit(bar(OF));
                    }
                    if (j < count) issue_s(0, ks);
                    if (j > 0) {
                        if (two) {
                            if (!(good = wait(bar(PF + 1), phase1++))) break;
                            tc_fence_after();
                            issue_o(1, vs, j > 1);
                            if (j == count) tc_commit(bar(OF + 1));
                        }
                        tc_commit(bar((kFp8 ? VE : TE) + vs));
                    }
                    if (j < count) {
                        if (two) issue_s(1, ks);
                        tc_commit(bar(TE + ks));
                        ++it;
                    }
                }
                if (!good) break;
            }
            ctl.left[0] = items0, ctl.left[1] = items1;
        } else if (warp == 2 && lane == 0) {
            // ================= what the issuer need not wait for itself =================
            // A wait costs it 150 to 250 clocks even where nothing is waited for.  So this thread
            // follows the tiles, in their order, and arrives with the first half's weights.
            uint32_t it = 0, edges = 0;
            for (int k = 0;; ++k) {
                const int b = k & 1;
                if (!wait(bar(MF + b), k >> 1)) break;
                const Item &item = ctl.item[b];
                if (!item.live) break;
                const int count = item.c1 - item.c0, edge = kFp8 ? INT_MAX : item.edge - item.c0;
                const auto keys = [&](uint32_t i) {
                    return kFp8 ? wait(bar(TF + i % kRingK), i / kRingK) : wait(bar(TF + 2 * i % kRingBf16), 2 * i / kRingBf16);
                };
                bool good = true;                        // the item's first K is the issuer's to wait for
                for (int j = 0; j < count && good; ++j, ++it) {
                    const uint32_t x = 2 * it + 1;
                    if (j >= edge) {
                        good = wait(bar(GE + edges % kUnclean), edges / kUnclean);
                        ++edges;
                    } else {
                        good = kFp8 ? wait(bar(VF + (it & 1)), it >> 1) : wait(bar(TF + x % kRingBf16), x / kRingBf16);
                    }
                    if (good && j + 1 < count) good = keys(it + 1);
                    if (good && it) good = wait(bar(PF), it - 1);        // one arrival a phase
                    if (good) mbar_arrive(bar(PF));
                }
                if (!good) break;
                mbar_arrive(bar(ME + b));
            }
        } else if (warp == 3) {
            // ================= keys and values =================
            const int box = a.c.page_size < kBlock ? a.c.page_size : kBlock, boxes = kBlock / box;     // rows of one; boxes of a block
            const int outside = a.c.num_pages * a.c.page_size;               // reads zeros
            uint32_t nt = 0, nk = 0, nx = 0, edges = 0;      // tiles of the ring (e4m3: of K, staged ones of V), edge blocks
            for (int k = 0;; ++k) {
                const int b = k & 1;
                if (!__all_sync(~0u, wait(bar(MF + b), k >> 1))) break;
                const Item &item = ctl.item[b];
                if (!item.live) break;
                const int c0 = item.c0, count = item.c1 - c0, len = item.len, kv = item.kv, edge = item.edge;
                const int *table = a.block_table + (long long)item.r * a.max_pages;
                // the row of the caches where this lane's box of a block starts
                const auto look = [&](int j) {
                    const int tok = (c0 + j) * kBlock + (lane % boxes) * box;
                    if (j >= count || tok >= len) return outside;
                    const int page = table[tok / a.c.page_size];
                    if (page < 0 || page >= a.c.num_pages) {
                        set_status(a.status, FP_ERR_DEVICE_BOUNDS);
                        return outside;
                    }
                    return page * a.c.page_size + tok % a.c.page_size;
                };
                const auto copy = [&](const CUtensorMap *map, uint32_t dst, uint32_t full, int z) {
                    if (lane == 0) mbar_expect_tx(full, kFp8 ? kHalf : kTile);
                    __syncwarp();
                    if (lane < (kFp8 ? 1 : 2) * boxes)
                        tma_load_3d(dst + (lane / boxes) * kHalf + (lane % boxes) * box * 128, map, full, (lane / boxes) * 64, kv, z);
                    __syncwarp();
                };
                bool good = true;
                int z0 = look(0), z1 = look(1);
                if (!kFp8) {
                    for (int x = 0; x < 2 * count && good; ++x) {
                        const uint32_t slot = nt % kRingBf16;
                        if (!(good = nt < kRingBf16 || __all_sync(~0u, wait(bar(TE + slot), (nt / kRingBf16) ^ 1)))) break;
                        const bool v = x & 1, unclean = v && c0 + x / 2 >= edge;
                        if (unclean && lane == 0) mbar_arrive(bar(TF + slot));       // the issuer waits for the cleaners instead
                        copy(v ? &map_v : &map_k, base + kSmemK + slot * kTile, unclean ? bar(GF + edges % kUnclean) : bar(TF + slot), z0);
                        edges += unclean;
                        ++nt;
                        if (v) {
                            z0 = z1;
                            z1 = look(x / 2 + 2);
                        }
                    }
                } else {
                    // K0 K1 K2 V0 K3 V1 ...: V of block j behind K of block j + 2
                    int zv = z0, zw = z1;                    // of the next two V
                    for (int j = 0; j < count + 2 && good; ++j) {
                        const int z2 = look(j + 2);
                        if (j < count) {
                            const uint32_t slot = nk % kRingK;
                            if (!(good = nk < kRingK || __all_sync(~0u, wait(bar(TE + slot), (nk / kRingK) ^ 1)))) break;
                            copy(&map_k, base + kSmemK + slot * kHalf, bar(TF + slot), z0);
                            ++nk;
                        }
                        if (j >= 2) {
                            const uint32_t slot = nx & 1;
                            if (!(good = nx < 2 || __all_sync(~0u, wait(bar(GE + slot), (nx >> 1) ^ 1)))) break;
                            copy(&map_v, base + kSmemStage + slot * kHalf, bar(GF + slot), zv);
                            ++nx;
                            zv = zw;
                            zw = z0;
                        }
                        z0 = z1;
                        z1 = z2;
                    }
                }
                if (!good) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ME + b));
            }
            if (lane == 0) ctl.left[2] = kFp8 ? nk : nt, ctl.left[3] = kFp8 ? nx : edges;
        }
    } else if (warp < 8) {
        setmaxnreg_dec<kRegsLoad>();
        // ================= loaders: e4m3 values become fp16; bf16 ones are cleaned where some rows do not attend them
        const int lt = tid - 128;
        uint32_t nv = 0, edges = 0;                      // blocks, edge blocks
        for (int k = 0; !dead; ++k) {
            const int b = k & 1;
            const bool got = wait.through_item(bar(MF + b), k >> 1);
            if (!__all_sync(~0u, got)) break;
            Item &item = ctl.item[b];
            if (!item.live) break;
            const int c0 = item.c0, count = item.c1 - c0, len = item.len, edge = item.edge, min_keys = item.min_keys;
            bool good = true;
            for (int j = kFp8 ? 0 : max(0, edge - c0); j < count && good; ++j) {
                if (!kFp8) {
                    const uint32_t tile = base + kSmemK + ((2 * (nv + j) + 1) % kRingBf16) * kTile;
                    if (!(good = __all_sync(~0u, wait.through_item(bar(GF + edges % kUnclean), edges / kUnclean)))) break;
                    const int key = (c0 + j) * kBlock + lt;         // a thread a row; can pass 2^31 behind the last token
                    if ((uint32_t)key >= (uint32_t)len) {
#pragma unroll 4
                        for (int p = 0; p < 16; ++p) st_shared_v4(piece_at(tile, lt, p), make_uint4(0, 0, 0, 0));
                    } else if (key >= min_keys) {
#pragma unroll 2
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
                    mbar_arrive(bar(GE + edges % kUnclean));
                    ++edges;
                } else {
                    const uint32_t s = nv & 1, tile = base + kSmemV + s * kTile;
                    if (!(good = nv < 2 || __all_sync(~0u, wait(bar(VE + s), (nv >> 1) ^ 1)))) break;
                    if (!(good = __all_sync(~0u, wait(bar(GF + s), nv >> 1)))) break;      // the staging ring goes as V's does
                    // rows 16 p + lt / 8, dims 16 c ..
                    const uint32_t from = base + kSmemStage + s * kHalf + lt * 16;
                    const int row0 = lt >> 3, c = lt & 7, o = c >> 2;
                    const auto convert = [&](uint4 w, uint32_t (&h)[8]) {
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) h[e] = halves_of(u[e >> 1] >> (16 * (e & 1)));
                    };
                    // lanes 4 .. 7 of a row write their two pieces the other way round: all banks, once
                    const auto put = [&](int row, const uint32_t (&h)[8]) {
                        const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
                        st_shared_v4(piece_at(tile, row, 2 * c + o), o ? hi : lo);
                        st_shared_v4(piece_at(tile, row, 2 * c + 1 - o), o ? lo : hi);
                    };
                    if (c0 + j < edge) {
#pragma unroll 1
                        for (int p = 0; p < 8; p += 2) {
                            uint4 w[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) w[i] = ld_shared_v4(from + (p + i) * 2048);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
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
                    mbar_arrive(bar(GE + s));
                    ++nv;
                }
            }
            if (!kFp8) nv += count;
            if (!__all_sync(~0u, good)) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(ME + b));
        }
    } else {
        setmaxnreg_inc<kRegsSoftmax>();
        // ================= softmax, a warpgroup a half, a thread a row =================
        const int t = (warp - 8) / 4, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t s_at = tmem + ((uint32_t)(quarter * 32) << 16) + t * 256, o_at = s_at + 128;
        const int own = row / a.g;                       // query of the half
        uint32_t phase = 0, items = 0;
        for (int k = 0; !dead; ++k) {
            const int b = k & 1;
            const bool got = wait.through_item(bar(MF + b), k >> 1);
            if (!__all_sync(~0u, got)) break;
            const Item &item = ctl.item[b];
            if (!item.live) break;
            const int i0 = 2 * a.half * item.tile + t * a.half, i = i0 + own, head = item.kv * a.g + row - own * a.g;
            const bool valid = own < a.half && i < item.rows;
            if (item.len && item.rows <= i0) {           // no row in this half
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ME + b));
                continue;
            }
            // a row that is none attends all with logits of 0, whatever its queries' place holds: masking it would
            // cost its warp the masks of every block
            const int keys = valid ? max(0, min(item.len, item.len - item.lq + i + 1)) : INT_MAX;
            const long long out_row = item.row0 + i;
            float cs = a.scale * kLog2e;                             // base-2 logits
            if (kFp8) cs *= __ldg(a.k_scale + item.kv);
            if (!valid) cs = 0.f;
            else if (a.q_scale) cs *= __ldg(a.q_scale + head);
            else if (kFp8) cs *= pow2f(-a.q_exponent[out_row * a.h_q + head]);
            const int count = item.c1 - item.c0, key0 = item.c0 * kBlock;
            // A weight is 2^(by x + off), up to 2^kTop where the maximum is set, and stands for 2^(cs x - m).  Products
            // are not rounded before `off` is added to them, so m is, up: by less than 8 below 2^27.  From there on,
            // where fp32 holds logits to 8 at best, weights go by half of cs' power of two, whose products with x are
            // exact, with 1 for the largest.  (Products rounded by an operation of their own took 5 to 9 %.)
            // next: what is added to by x to see whether the maximum follows; all but -inf does at first
            float m = -INFINITY, l = 0.f, by = cs, off = 0.f, next = INFINITY;
            bool ok = true;
            for (int j = 0; j < count; ++j, ++phase) {
                const bool there = wait(bar(SF + t), phase);
                if (!__all_sync(~0u, there)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
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
                const bool grow = fmaf(raw, by, next) > kTop + kSlack;
                const bool any_grow = __any_sync(~0u, grow);
                float keep = 1.f;
                if (grow) {
                    const float near = __fmaf_ru(raw, cs, -kTop);
                    const bool far = fabsf(near) >= 0x1p27f;
                    const float to = far ? raw * cs : near;
                    by = far ? 0.5f * __int_as_float(__float_as_int(cs) & 0x7f800000) : cs;
                    next = off = far ? -raw * by : -to;
                    keep = fast_exp2(m - to);                        // 0 for the first
                    m = to;
                    l *= keep;
                }
                const uint64_t cc = f2_pack(by, by), oo = f2_pack(off, off);
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
            if (count > 0) {
                const bool done = wait(bar(OF + t), items);
                if (!__all_sync(~0u, done)) break;
                tc_fence_after();
                ++items;
            }
            const bool whole = item.opens && item.closes;
            const float v_scale = kFp8 ? __ldg(a.v_scale + item.kv) : 1.f;
            const float out_by = !whole ? v_scale : l == 0.f ? 0.f : v_scale / l;
            const int not_finite = *reinterpret_cast<const volatile int *>(&item.not_finite);
            const long long slot = (long long)blockIdx.x * 2 + (item.opens ? 1 : 0);
            if (item.len == 0) {                         // all rows of the request: half a warp each
                const int lane16 = lane & 15, from = 2 * (warp - 8) + (lane >> 4);
#pragma unroll 4
                for (int r = from; r < item.rows * a.g; r += 16) {
                    const int j = r / item.rows, at = item.row0 + r - j * item.rows, h = item.kv * a.g + j;
                    reinterpret_cast<uint4 *>(a.out + ((long long)at * a.h_q + h) * kHeadDim)[lane16] = make_uint4(0, 0, 0, 0);
                    if (a.lse && lane16 == 0) a.lse[(long long)h * a.total_q + at] = -INFINITY;
                }
            }
            const unsigned long long mine = valid ? (unsigned long long)(a.out + (out_row * a.h_q + head) * kHeadDim) : 0;
#pragma unroll 1
            for (int c = 0; c < 4 && item.len; ++c) {
                uint32_t o[32];
                if (count > 0) {
                    tmem_ld32(o_at + c * 32, o);
                    tmem_ld_wait();
                    reg_fence(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * out_by);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0;
                }
                if (not_finite)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (item.from[32 * c + e] < keys) o[e] = 0x7fffffffu;
                if (whole) {
                    // 64 bytes of a row each: four lanes swap pieces, so that they write a row together
                    // and not 16 bytes of a row of their own each
                    uint32_t w[4][4];                    // [piece][word]
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e / 4][e % 4] = pack16<false>(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
#pragma unroll
                    for (int d = 1; d <= 2; d *= 2) {
                        const bool up = lane & d;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            if (x & d) continue;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t got = __shfl_xor_sync(~0u, up ? w[x][e] : w[x | d][e], d);
                                if (up) w[x][e] = got; else w[x | d][e] = got;
                            }
                        }
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {        // piece lane % 4 of the row of lane (lane & ~3) + x
                        const unsigned long long to = __shfl_sync(~0u, mine, (lane & ~3) + x);
                        if (to) reinterpret_cast<uint4 *>(to)[4 * c + (lane & 3)] = make_uint4(w[x][0], w[x][1], w[x][2], w[x][3]);
                    }
                } else {                                 // [4 dims][row], rows side by side
                    uint4 *to = reinterpret_cast<uint4 *>(sc.o) + (slot * 32 + 8 * c) * kRows + t * kBlock + row;
#pragma unroll
                    for (int e = 0; e < 8; ++e) to[e * kRows] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
            }
            if (!whole) sc.ml[slot * kRows + t * kBlock + row] = make_float2(m, l);
            else if (valid && a.lse && item.len) a.lse[(long long)head * a.total_q + out_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            // the next item's first product over O follows its weights, which follow these reads
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(ME + b));
        }
    }
    tc_fence_before();
    __syncthreads();
    // Nothing is on its way when the block leaves: products and their arrivals on barriers, and after a stop the
    // copies armed last.  Here all roles have left, so that none gives up after another has looked.
    if (tid == 0 && !dead) {
        tc_commit(bar(DR));
        mbar_wait_drain(bar(DR), 0);
        if (ld_shared_volatile(wait.abort)) {
            for (int t = 0; t < 2; ++t)
                if (ctl.left[t]) mbar_wait_drain(bar(QF + t), (ctl.left[t] - 1) & 1);
            constexpr uint32_t kRing = kFp8 ? kRingK : kRingBf16, kStaged = kFp8 ? 2 : kUnclean;
            const uint32_t m = ctl.left[2], g = ctl.left[3];
            for (uint32_t i = m < kRing ? 0 : m - kRing; i < m; ++i) mbar_wait_drain(bar(TF + i % kRing), (i / kRing) & 1);
            for (uint32_t i = g < kStaged ? 0 : g - kStaged; i < g; ++i) mbar_wait_drain(bar(GF + i % kStaged), (i / kStaged) & 1);
        }
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Queries of another type than the tiles take, for the copies to fetch: e4m3 ones as bf16
// rows; bf16 ones of an e4m3 cache as two e4m3 terms, [2][total_q, h_q, 128] codes, the
// exponents of their powers of two behind them.  16 lanes a row.
template <bool kTerms>
__global__ void __launch_bounds__(256) queries_kernel(PAttn a, void *to, signed char *exponent) {
    after_previous();
    const long long rows = (long long)a.total_q * a.h_q, row = blockIdx.x * 16ll + threadIdx.x / 16;
    const int c = threadIdx.x & 15;
    if (row >= rows) return;                             // 16 lanes together
    const long long tok = row / a.h_q, at = tok * a.q_stride_tok + (row - tok * a.h_q) * a.q_stride_head + 8 * c;
    if (!kTerms) {
        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const unsigned char *>(a.q) + at);
        const uint32_t h[4] = {bf16_of(w.x), bf16_of(w.x >> 16), bf16_of(w.y), bf16_of(w.y >> 16)};
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(to) + row * kHeadDim + 8 * c) = make_uint4(h[0], h[1], h[2], h[3]);
        return;
    }
    const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + at);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    float x[8], top = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(v[e] << 16);
        x[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
        top = max3f(top, fabsf(x[2 * e]), fabsf(x[2 * e + 1]));
    }
    const unsigned lanes = 0xffffu << (threadIdx.x & 16);
#pragma unroll
    for (int d = 1; d < 16; d *= 2) top = fmaxf(top, __shfl_xor_sync(lanes, top, d));
    const int ex = term_exp(top);
    const float up = pow2f(ex);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const TwoTerms z = two_terms(x[2 * e], x[2 * e + 1], up);
        hi[e] = z.hi;
        lo[e] = z.lo;
    }
    unsigned char *p = static_cast<unsigned char *>(to) + row * kHeadDim + 8 * c;
    *reinterpret_cast<uint2 *>(p) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
    *reinterpret_cast<uint2 *>(p + rows * kHeadDim) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
    if (c == 0) exponent[row] = (signed char)ex;
}

__global__ void wait_timeout_kernel(int *status, unsigned long long limit_ns) {
    __shared__ __align__(8) unsigned long long nothing;
    __shared__ uint32_t abort;
    abort = 0;
    mbar_init(smem_u32(&nothing), 1);
    fence_barrier_init();
    Waits{smem_u32(&abort), status, limit_ns, limit_ns}(smem_u32(&nothing), 0);
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
// [n2][n1][128] of bf16 or e4m3 at strides s1, s2 (elements): boxes of 128 bytes of a row by b1
// by b2, swizzled as the products take them or plain; past the end it reads zeros.
bool make_map(CUtensorMap *m, const void *base, long long n1, long long n2, long long s1, long long s2, int b1, int b2, bool fp8,
              bool swizzled) {
    const EncodeFn fn = encode();
    if (!fn) return false;
    const cuuint64_t esz = fp8 ? 1 : 2;
    const cuuint64_t dims[3] = {kHeadDim, (cuuint64_t)n1, (cuuint64_t)n2};
    const cuuint64_t strides[2] = {(cuuint64_t)s1 * esz, (cuuint64_t)s2 * esz};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / esz), (cuuint32_t)b1, (cuuint32_t)b2};
    const cuuint32_t one[3] = {1, 1, 1};
    return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides,
              box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Thread blocks: one for each SM, and no more than the longest lengths that the table holds would use.
int tiles_blocks(const PAttn &a) {
    const long long rows = a.cu ? a.total_q : (long long)a.batch * a.max_q;
    const double items = (double)a.c.h_kv * ((double)rows / (2 * (kBlock / a.g)) + a.batch);
    const double blocks = items * ((double)a.max_pages * a.c.page_size + 2 * kItemKeys) / (kBlock * kMinBlocks) + 1;
    return blocks < kSm ? (int)blocks : kSm;
}

// Joins the parts of the items that several blocks share: part 0 in the first block's second
// slot, the others in the first slots of the blocks behind it.  A task is 8 rows of an open
// item; a lane has every fourth piece of 4 dims of one.  Where there are few tasks a block
// takes one, its warps a share of the parts each; else a warp does.
__global__ void __launch_bounds__(kJoinWarps * 32) tiles_join_kernel(PAttn a, Scratch sc, int blocks) {
    __shared__ Open list[kSm];
    __shared__ int first[kSm];
    __shared__ int opens_in[kJoinWarps];
    __shared__ float4 part_o[kJoinWarps][8][32];
    __shared__ float part_l[kJoinWarps][32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    after_previous();
    let_next();
    static_assert(kSm <= kJoinWarps * 32, "a thread for each block");
    Open rec;
    rec.parts = 0;
    if ((int)threadIdx.x < blocks) rec = sc.open[threadIdx.x];
    const unsigned vote = __ballot_sync(~0u, rec.parts > 0);
    if (lane == 0) opens_in[warp] = __popc(vote);
    __syncthreads();
    int opens = 0, at = __popc(vote & ((1u << lane) - 1));
    for (int w = 0; w < kJoinWarps; ++w) {
        if (w < warp) at += opens_in[w];
        opens += opens_in[w];
    }
    if (rec.parts > 0) {
        list[at] = rec;
        first[at] = threadIdx.x;
    }
    __syncthreads();
    const int tasks = opens * (kRows / 8), row8 = lane & 7, piece0 = lane >> 3;
    const bool wide = tasks <= (int)gridDim.x;
    const int step = wide ? 1 : kJoinWarps;
    for (int task0 = blockIdx.x * step; task0 < tasks; task0 += gridDim.x * step) {
        const int task = task0 + (wide ? 0 : warp);
        const bool live = task < tasks;
        const Open it = list[live ? task / (kRows / 8) : 0];
        const int b = first[live ? task / (kRows / 8) : 0], row = task % (kRows / 8) * 8 + row8;
        const int in_half = row & (kBlock - 1), own = in_half / a.g, i = (2 * it.tile + row / kBlock) * a.half + own;
        const bool there = live && own < a.half && i < it.rows;
        float top = -INFINITY, l = 0.f;
        float4 o[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (__any_sync(~0u, there)) {
            const auto slot = [&](int p) { return (long long)(b + p) * 2 + (p == 0); };
            for (int p = piece0; p < it.parts; p += 4) top = fmaxf(top, sc.ml[slot(p) * kRows + row].x);
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
            for (int p = wide ? warp : 0; p < it.parts; p += wide ? kJoinWarps : 1) {
                const float2 e = sc.ml[slot(p) * kRows + row];
                const float4 *from = reinterpret_cast<const float4 *>(sc.o) + (slot(p) * 32 + piece0) * kRows + row;
                float4 v[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) v[x] = from[4 * x * kRows];
                const float f = e.x == -INFINITY ? 0.f : exp2f(e.x - top);
                l += e.x == -INFINITY ? e.y : f * e.y;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    o[x].x = fmaf(f, v[x].x, o[x].x);
                    o[x].y = fmaf(f, v[x].y, o[x].y);
                    o[x].z = fmaf(f, v[x].z, o[x].z);
                    o[x].w = fmaf(f, v[x].w, o[x].w);
                }
            }
        }
        if (wide) {
#pragma unroll
            for (int x = 0; x < 8; ++x) part_o[warp][x][lane] = o[x];
            part_l[warp][lane] = l;
            __syncthreads();
            if (warp == 0)
                for (int w = 1; w < kJoinWarps; ++w) {
                    l += part_l[w][lane];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const float4 v = part_o[w][x][lane];
                        o[x].x += v.x, o[x].y += v.y, o[x].z += v.z, o[x].w += v.w;
                    }
                }
        }
        if (there && !(wide && warp)) {
            const int head = it.kv * a.g + in_half - own * a.g;
            const long long out_row = it.row0 + i;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint2 *to = reinterpret_cast<uint2 *>(a.out + (out_row * a.h_q + head) * kHeadDim) + piece0;
#pragma unroll
            for (int x = 0; x < 8; ++x)
                to[4 * x] = make_uint2(pack16<false>(o[x].x * inv, o[x].y * inv), pack16<false>(o[x].z * inv, o[x].w * inv));
            if (a.lse && piece0 == 0) a.lse[(long long)head * a.total_q + out_row] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
        }
        if (wide) __syncthreads();
    }
}

// Bytes that queries of another type take (queries_kernel).
size_t converted_bytes(const PAttn &a) {
    const size_t rows = (size_t)a.total_q * a.h_q;
    return (a.k_scale != nullptr) == a.q_codes ? 0 : align256(rows * 2 * kHeadDim) + align256(rows);
}

}  // namespace

size_t cache_tiles_scratch_bytes(const PAttn &a) {
    const size_t n = tiles_blocks(a);
    return align256(n * sizeof(Open)) + align256(n * 2 * kRows * sizeof(float2)) + n * 2 * kRows * kHeadDim * sizeof(float) +
           converted_bytes(a);
}

cudaError_t launch_cache_wait_timeout(int *status, unsigned long long limit_ns, cudaStream_t st) {
    wait_timeout_kernel<<<1, 1, 0, st>>>(status, limit_ns);
    return cudaGetLastError();
}

cudaError_t launch_cache_tiles(const PAttn &args, void *scratch, unsigned long long limit_ns, cudaStream_t st) {
    PAttn a = args;
    a.half = kBlock / a.g;
    const size_t n = tiles_blocks(a);
    char *p = static_cast<char *>(scratch);
    Scratch sc;
    sc.open = reinterpret_cast<Open *>(p);
    p += align256(n * sizeof(Open));
    sc.ml = reinterpret_cast<float2 *>(p);
    p += align256(n * 2 * kRows * sizeof(float2));
    sc.o = reinterpret_cast<float *>(p);
    p += n * 2 * kRows * kHeadDim * sizeof(float);
    const bool fp8 = a.k_scale != nullptr;
    const long long rows = (long long)a.total_q * a.h_q;
    const void *q = a.q;
    long long q_tok = a.q_stride_tok, q_head = a.q_stride_head, q_rows = a.total_q;
    cudaError_t e;
    if (converted_bytes(a)) {
        signed char *exponent = reinterpret_cast<signed char *>(p + align256((size_t)rows * 2 * kHeadDim));
        const auto kernel = fp8 ? queries_kernel<true> : queries_kernel<false>;
        if ((e = launch_chained(kernel, (unsigned)((rows + 15) / 16), 256, 0, st, a, (void *)p, exponent)) != cudaSuccess) return e;
        q = p;
        q_head = kHeadDim;
        q_tok = (long long)a.h_q * kHeadDim;
        if (fp8) {
            q_rows = 2ll * a.total_q;
            a.q_exponent = exponent;
        }
    }
    CUtensorMap map_q, map_k, map_v;
    const Pages &c = a.c;
    const long long tokens = (long long)c.num_pages * c.page_size, pitch = (long long)c.h_kv * kHeadDim;
    const int box = c.page_size < kBlock ? c.page_size : kBlock;
    if (!make_map(&map_q, q, a.h_q, q_rows, q_head, q_tok, a.g, a.half, fp8, true) ||
        !make_map(&map_k, c.k, c.h_kv, tokens, kHeadDim, pitch, 1, box, fp8, true) ||
        !make_map(&map_v, c.v, c.h_kv, tokens, kHeadDim, pitch, 1, box, fp8, !fp8))
        return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> told[2];
    const unsigned long long item_ns = kBlockNs * ((unsigned long long)(a.max_len + rows / c.h_kv) / kBlock + 1);
    const unsigned long long item_limit_ns = limit_ns + item_ns < limit_ns ? ~0ull : limit_ns + item_ns;
    if ((e = launch_large(told[fp8], fp8 ? tiles_kernel<true> : tiles_kernel<false>, (unsigned)n, kTilesThreads, kSmem, st, a, sc,
                          map_q, map_k, map_v, limit_ns, item_limit_ns)) != cudaSuccess)
        return e;
    return launch_chained(tiles_join_kernel, (unsigned)n * 4, kJoinWarps * 32, 0, st, a, sc, (int)n);
}

}  // namespace fp
