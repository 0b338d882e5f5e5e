// fp_cache_attn: attention over the bf16 / e4m3 paged cache at any position, by columns.
//
// A column is one (query, head) of a kv head's group, and keys fill the long side of
// m16n8k16 products, so that a decode step of up to 8 query heads a kv head pads nothing:
//   S^T[key, col] = K Q^T,   O^T[dim, col] = V^T P^T.
// K and V^T fragments come out of shared memory by ldmatrix, and the weights become the
// second product's operand by an 8 x 8 transpose in registers.
// A bf16 cache takes bf16 operands: queries as they are (e4m3 ones exactly), weights rounded
// to bf16 (2^-8 of each).  Of an e4m3 cache K's codes are multiplied as they are (m16n8k32),
// with e4m3 queries, or with bf16 ones under a power of two as two e4m3 terms of 4 bits each,
// which hold 8 bits exactly down to 2^-9 of the row's largest, and the rest to 2^-17 of it;
// V's become fp16, exactly, in registers, weights fp16 (2^-11).
// For V^T two keys of a dim have to meet in a register: the 16-bit transpose brings two dims
// of two keys, which a byte permutation sorts, and a tile's rows stand for even, then odd dims.
//
// Weights are exp2(logit - m + 10), m a maximum that only follows when the logits pass it by
// 4 (a warp vote), so that the largest weight so far is between 2^10 and 2^14 and fp16 loses
// nothing above 2^-34 of it.  Sums, maxima and outputs are fp32.
//
// Work is cut as in the attention over the 4-bit cache: the (request, kv head, column tile)
// items laid end to end in chunks of 16 tokens, cut into equal ranges, one a thread block;
// the warps of a block take every kWarps-th chunk through rings of their own (cp.async) and
// join at the item's end; an item that a range's end cuts is joined by a second kernel.
//
// Bounds.  One octet of columns: memory.  64 requests up to 16384 (32/4 heads, bf16, 1.07 GB)
// 165 us, 6.5 TB/s, 0.96 of the measured copy rate; e4m3 0.76 to 0.87 of it, by the box (262144
// tokens of 8 heads, 537 MB, 91 to 104 us), where taking V's codes apart fills 44 % of the issue slots.  More octets: latency,
// of 8 warps an SM (255 registers): 32 requests up to 8192 with 1 to 8 tokens of 4 heads (up to 4
// octets, 530 MB) 100 us, 0.78.
#include <limits.h>

#include <type_traits>

#include "cache.cuh"
#include "device_lengths.cuh"

namespace fp {
namespace {

constexpr int kMinChunks = 2 * kWarps;       // least work worth a thread block
// What starting and ending an item costs, in chunks, and what a chunk costs by the octets in use
// (bf16 more for its bytes, e4m3 for its instructions).  32 requests up to 8192 of 1 to 8 tokens
// (32/8 heads), us with items of 8 + 2 octets, 16 + 4, 24 + 6 chunks: bf16 116, 101, 101; e4m3 of
// 14 + 2, 28 + 4, 40 + 6: 123, 128, 134; with 1, 2, 4, 10 for a chunk without octets e4m3 131, 123,
// 130, 137.
template <bool kFp8, int NT>
constexpr int item_chunks() { return kFp8 ? 14 + 2 * NT : 16 + 4 * NT; }
template <bool kFp8, int NT>
__device__ __forceinline__ int chunk_units(int octets) { return NT == 1 ? 1 : (kFp8 ? 2 : 4) + octets; }
// Longest cache, by the width of its table, that is not cut (one launch instead of two).
constexpr int kWholeChunks = 64;

template <bool kFp8>
constexpr int row_bytes() { return kFp8 ? kHeadDim : 2 * kHeadDim; }
template <bool kFp8>
constexpr int chunk_bytes() { return 2 * kChunk * row_bytes<kFp8>(); }
template <bool kFp8, int NT>
constexpr int blocks_per_sm() { return NT == 1 && kFp8 ? 3 : 2; }
template <bool kFp8, int NT>
constexpr int stages() { return kFp8 && NT > 1 ? 6 : 3; }
template <bool kFp8>
constexpr int most_blocks() { return kSm * blocks_per_sm<kFp8, 1>(); }

// What a page id out of range, or an empty cache, reads.
__device__ __align__(16) unsigned char zero_row[256];

template <bool kFp8>
__device__ __forceinline__ void mma16(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    if (kFp8)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 32 dims of e4m3 codes: a register holds four, as ldmatrix brings them.
__device__ __forceinline__ void mma32(float c[4], const uint32_t a[4], uint2 b) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ void load4(uint32_t r[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void load4_transposed(uint32_t r[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
// The top bit of each half that is an infinity or a NaN.
template <bool kFp8>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    return ((w & 0x7fff7fffu) + (kFp8 ? 0x04000400u : 0x00800080u)) & 0x80008000u;
}

// What one lane holds of 8 columns: queries as B fragments of 8 steps of 16 dims -- for an e4m3
// cache of 4 steps of 32, and the second terms' behind them -- and what a column's products have
// to be scaled by to be base-2 logits.
struct Queries {
    uint2 f[8];
    float factor;              // of column lane / 4
};
// A column's 32 elements of this lane, and its scale: dims 16 s + 2 j4 + {0, 1, 8, 9}, or for
// an e4m3 cache 16 s + 4 j4 + {0, 1, 2, 3}; e4m3 codes as two bytes a word, or four.
struct RawQuery {
    uint2 w[8];
    float scale;
};

template <bool kFp8>
__device__ __forceinline__ RawQuery fetch_query(const PAttn &a, const Request &q, int kv, int col) {
    const int j4 = threadIdx.x & 3, i = col / a.g, head = kv * a.g + col % a.g;
    RawQuery raw;
    raw.scale = a.scale * kLog2e;
    if (kFp8) raw.scale *= a.k_scale[kv];
#pragma unroll
    for (int s = 0; s < 8; ++s) raw.w[s] = make_uint2(0, 0);
    if (i < q.rows) {
        const long long at = (q.row0 + i) * a.q_stride_tok + head * a.q_stride_head + (kFp8 ? 4 : 2) * j4;
        if (a.q_scale) {
            raw.scale *= a.q_scale[head];
            const unsigned char *p = static_cast<const unsigned char *>(a.q) + at;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                if (kFp8)
                    raw.w[s].x = *reinterpret_cast<const uint32_t *>(p + 16 * s);
                else
                    raw.w[s] = make_uint2(*reinterpret_cast<const uint16_t *>(p + 16 * s),
                                          *reinterpret_cast<const uint16_t *>(p + 16 * s + 8));
            }
        } else {
            const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(a.q) + at;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                if (kFp8)
                    raw.w[s] = *reinterpret_cast<const uint2 *>(p + 16 * s);
                else
                    raw.w[s] = make_uint2(*reinterpret_cast<const uint32_t *>(p + 16 * s),
                                          *reinterpret_cast<const uint32_t *>(p + 16 * s + 8));
            }
        }
    }
    return raw;
}

template <bool kFp8>
__device__ __forceinline__ void make_queries(const RawQuery &raw, bool e4m3, Queries &out) {
    out.factor = raw.scale;
    if (kFp8 && e4m3) {
#pragma unroll
        for (int s = 0; s < 4; ++s) out.f[s] = make_uint2(raw.w[2 * s].x, raw.w[2 * s + 1].x);
    } else if (e4m3) {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            out.f[s] = make_uint2(bf16_of(raw.w[s].x), bf16_of(raw.w[s].y));
        }
    } else if (!kFp8) {
#pragma unroll
        for (int s = 0; s < 8; ++s) out.f[s] = raw.w[s];
    } else {
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t w = e ? raw.w[s].y : raw.w[s].x;
                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u))));
            }
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        const int ex = term_exp(top);
        const float up = pow2f(ex);
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            uint32_t term[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t w = e ? raw.w[s].y : raw.w[s].x;
                const TwoTerms z = two_terms(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u), up);
                term[0] |= z.hi << 16 * e;
                term[1] |= z.lo << 16 * e;
            }
            (s & 1 ? out.f[s / 2].y : out.f[s / 2].x) = term[0];
            (s & 1 ? out.f[4 + s / 2].y : out.f[4 + s / 2].x) = term[1];
        }
        out.factor *= pow2f(-ex);
    }
}

template <bool kFp8, int NT>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<kFp8, NT>()) columns_kernel(PAttn a, Scratch sc) {
    constexpr int kCols = 8 * NT, kRow = row_bytes<kFp8>(), kBytes = chunk_bytes<kFp8>(), kStages = stages<kFp8, NT>();
    constexpr int kRing = kStages * kBytes, kItem = item_chunks<kFp8, NT>();
    constexpr int kRowLanes = kRow / 16, kRowsAt = 32 / kRowLanes;     // lanes that copy a row, rows copied at once
    constexpr bool kSharedQ = NT > 1;          // queries' fragments in shared memory instead of registers
    extern __shared__ __align__(128) unsigned char smem_raw[];
    __shared__ long long warp_sums[kWarps];
    __shared__ long long s_at;
    __shared__ int s_r;
    __shared__ Request s_q;
    __shared__ float2 ml[kWarps][kCols];
    __shared__ uint2 s_frag[kSharedQ ? NT : 1][8][32];
    __shared__ float s_factor[kSharedQ ? kCols : 1];
    after_previous();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31, r8 = lane >> 2, j4 = lane & 3;

    // this block's range of units, and the request it starts in: an item is its start and
    // end, then its chunks
    const auto tiles_of_columns = [&](const Request &q) {
        return (long long)q.rows * a.g > a.most_columns ? 0 : tiles_of(a, q, kCols);
    };
    const auto octets_of = [&](const Request &q, int tile) { return (min(kCols, q.rows * a.g - tile * kCols) + 7) / 8; };
    const auto units = [&](const Request &q) {
        const int tiles = tiles_of_columns(q);
        if (tiles == 0 || a.whole) return (long long)a.c.h_kv * tiles;
        return (long long)a.c.h_kv * (kItem + chunks_of(q)) *
               ((tiles - 1) * chunk_units<kFp8, NT>(NT) + chunk_units<kFp8, NT>(octets_of(q, tiles - 1)));
    };
    const int each = (a.batch + kThreads - 1) / kThreads;      // requests a thread adds up
    Request q = {0, 0, 0, 0};
    long long n = 0, total;
    for (int r = tid * each; r < min(a.batch, (tid + 1) * each); ++r) n += units(q = request_of(a, r));
    long long low = block_scan(n, &total, warp_sums);
    const long long want = a.whole ? total : total / (kMinChunks * chunk_units<kFp8, NT>(NT)) + 1;
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
    int tiles = tiles_of_columns(q), chunks = chunks_of(q);
    int kv, tile;                                 // of the current item
    {
        const long long full = a.whole ? 1 : (long long)(kItem + chunks) * chunk_units<kFp8, NT>(NT);
        const long long last = a.whole ? 1 : (long long)(kItem + chunks) * chunk_units<kFp8, NT>(octets_of(q, tiles - 1));
        const long long head = (tiles - 1) * full + last;
        kv = (int)quotient(first - item0, head);
        item0 += kv * head;
        tile = min((int)quotient(first - item0, full), tiles - 1);
        item0 += tile * full;
    }
    // 256-byte aligned, so that a piece's number is XORed inside its row
    unsigned char *smem = smem_raw + (-smem_addr(smem_raw) & 255u), *ring = smem + warp * kRing;
    const uint32_t ring_at = smem_addr(ring);
    const int per_page = a.c.page_size / kChunk;
    const long long pitch = (long long)a.c.h_kv * kRow;               // bytes from token to token
    // A row's 16-byte pieces lie in shared memory at their number XOR the row's (mod 8), so that the
    // eight rows of a matrix are in eight groups of banks.  Rows are copied kRowsAt at a time.
    const bool terms = a.q_scale == nullptr;      // e4m3 cache: two of each query
    const int copy_row = lane / kRowLanes, copy_piece = lane % kRowLanes;
    const uint32_t copy_at = copy_row * kRow + ((copy_piece ^ copy_row) << 4);
    // Matrices of a load: K rows 0-7 and 8-15 of one piece, then of the next; V (transposed) for bf16
    // the two pieces of rows 0-7, then of 8-15, for e4m3 as K.
    const int mat = lane >> 3, mat_row = (lane & 7) + 8 * (mat & 1), v_row = (lane & 7) + 8 * (kFp8 ? mat & 1 : mat >> 1);
    const uint32_t k_lane = mat_row * kRow + (((mat >> 1) ^ (lane & 7)) << 4);
    const uint32_t v_lane = kChunk * kRow + v_row * kRow + (((kFp8 ? mat >> 1 : mat & 1) ^ (lane & 7)) << 4);

    for (long long at = first; at < end;) {
        if (tile == tiles) {
            tile = 0;
            ++kv;
        }
        while (kv >= a.c.h_kv || tiles == 0) {    // the next request that has rows
            if (++r >= a.batch) return;           // lengths that changed under the kernel
            q = request_of(a, r);
            tiles = tiles_of_columns(q);
            chunks = chunks_of(q);
            kv = tile = 0;
        }
        const int octets = octets_of(q, tile), weight = chunk_units<kFp8, NT>(octets);
        const long long next = a.whole ? item0 + 1 : item0 + (long long)(kItem + chunks) * weight;
        const int c0 = a.whole ? 0 : max(0, (int)((uint32_t)(at - item0) / weight) - kItem);    // an item is below 2^31 units
        const int c1 = a.whole ? chunks : max(0, (int)((uint32_t)(min(end, next) - item0) / weight) - kItem);
        if (c1 <= c0) {                           // the range ends inside the item's start
            at = item0 = next;
            ++tile;
            continue;
        }
        const int mine = c1 - c0 > warp ? (c1 - c0 - warp + kWarps - 1) / kWarps : 0;

        // -- copies ahead: chunk c0 + warp + i * kWarps into stage i % kStages.  Lane l
        //    looks up the addresses of chunks l, l + 32, ...
        long long src = -1;                       // byte offset of the chunk in either cache, -1: zeros
        int page = -1, in_page = 0;
        const auto look_up = [&](int i) {         // the page id of chunk i + lane ...
            const int c = c0 + warp + (i + lane) * kWarps, pg = c / per_page;
            page = i + lane < mine && q.len > 0 ? a.block_table[(long long)r * a.max_pages + pg] : -1;
            in_page = c - pg * per_page;
        };
        const auto locate = [&](int i) {          // ... and the chunk's place
            src = -1;
            if (page >= 0 && page < a.c.num_pages)
                src = ((long long)page * a.c.page_size + in_page * kChunk) * pitch + kv * kRow;
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
                const long long from = __shfl_sync(~0u, src, issued & 31);
                const uint32_t dst = ring_at + (issued % kStages) * kBytes + copy_at;
                const long long step = from < 0 ? 0 : pitch * kRowsAt;
                const long long off = from < 0 ? 0 : from + copy_row * pitch + copy_piece * 16;
                const unsigned char *pk = (from < 0 ? zero_row : a.c.k) + off, *pv = (from < 0 ? zero_row : a.c.v) + off;
#pragma unroll
                for (int i = 0; i < kChunk / kRowsAt; ++i) {
                    // rows kRowsAt * i + copy_row: XOR by the multiple is a XOR of its own bits
                    const uint32_t d = (dst + i * kRowsAt * kRow) ^ ((i * kRowsAt & 7) << 4);
                    copy16(d, pk + i * step);
                    copy16(d + kChunk * kRow, pv + i * step);
                }
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
            if (octet < NT) raw[t] = fetch_query<kFp8>(a, q, kv, tile * kCols + octet * 8 + r8);
        }
        locate(0);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue();
        Queries qs[kOwn];
#pragma unroll
        for (int t = 0; t < kOwn; ++t) {
            const int octet = kSharedQ ? t * kWarps + warp : t;
            if (octet >= NT) continue;            // whole warps
            make_queries<kFp8>(raw[t], a.q_scale != nullptr, qs[t]);
            if (kSharedQ) {
#pragma unroll
                for (int s = 0; s < 8; ++s) s_frag[octet][s][lane] = qs[t].f[s];
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
        float base[NT][2];                        // log2 of what weight 1 stands for (-inf: no key yet)
        float sum[NT][2];                         // this lane's share of the weights
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int m = 0; m < 8; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][m][e] = 0.f;
            base[t][0] = base[t][1] = -INFINITY;
            sum[t][0] = sum[t][1] = 0.f;
        }

        // octets: those of the tile in use (the others are left out)
        const auto step = [&](int i, auto edge, auto octets) {
            constexpr bool kEdge = decltype(edge)::value;
            constexpr int L = decltype(octets)::value;
            copies_wait<kStages - 2>();
            __syncwarp();
            issue();
            const uint32_t chunk = ring_at + (i % kStages) * kBytes;
            const int t0 = (c0 + warp + i * kWarps) * kChunk;

            // logits: rows r8 and r8 + 8, two columns each; one octet in two chains of products
            constexpr int kChains = L == 1 ? 2 : 1;
            float x[L * kChains][4];
#pragma unroll
            for (int t = 0; t < L * kChains; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[t][e] = 0.f;
#pragma unroll
            for (int s = 0; s < (kFp8 ? 4 : 8); ++s) {
                uint32_t w[4];
                load4(w, (chunk + k_lane) ^ (s << 5));
#pragma unroll
                for (int t = 0; t < L; ++t) {
                    const auto query = [&](int i) { return kSharedQ ? s_frag[t][i][lane] : qs[kSharedQ ? 0 : t].f[i]; };
                    float *sums = x[kChains == 2 ? s & 1 : t];
                    if (kFp8) {
                        mma32(sums, w, query(s));
                        if (terms) mma32(sums, w, query(4 + s));
                    } else {
                        const uint2 f = query(s);
                        mma16<false>(sums, w, f.x, f.y);
                    }
                }
            }
            if (kChains == 2)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[0][e] += x[kChains - 1][e];

            // weights
            float y[L][4], top = -INFINITY;
#pragma unroll
            for (int t = 0; t < L; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[t][e] = fmaf(x[t][e], factor[t][e & 1], -base[t][e & 1]);
                    if (kEdge && t0 + r8 + 4 * (e & 2) >= keys_of(t, e & 1)) y[t][e] = -INFINITY;
                    top = fmaxf(top, y[t][e]);
                }
            if (__any_sync(~0u, top > kTop + kSlack)) {            // a maximum to follow
#pragma unroll
                for (int t = 0; t < L; ++t)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const bool out0 = y[t][c] == -INFINITY, out1 = y[t][c + 2] == -INFINITY;
                        const float l0 = out0 ? -INFINITY : x[t][c] * factor[t][c];
                        const float l1 = out1 ? -INFINITY : x[t][c + 2] * factor[t][c];
                        float m = fmaxf(l0, l1);
#pragma unroll
                        for (int d = 4; d < 32; d *= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
                        const float old = base[t][c], b = fmaxf(old, base_below(m));
                        const float keep = b == -INFINITY ? 1.f : exp2f(old - b);
                        base[t][c] = b;
                        sum[t][c] *= keep;
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
                sum[t][0] += y[t][0] + y[t][2];
                sum[t][1] += y[t][1] + y[t][3];
                p[t][0] = transpose8(pack16<kFp8>(y[t][0], y[t][1]));
                p[t][1] = transpose8(pack16<kFp8>(y[t][2], y[t][3]));
            }

            // values: tile m's registers hold keys 2 j4, 2 j4 + 1 (and 8 further) of its rows r8, r8 + 8
            uint32_t keep[2] = {~0u, ~0u}, late[2] = {0, 0};
            if (kEdge) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int tok = t0 + 8 * h + 2 * j4;
                    // behind the last token anything may lie ...
                    keep[h] = (tok < q.len ? 0xffffu : 0u) | (tok + 1 < q.len ? 0xffff0000u : 0u);
                    // ... and these some columns do not attend
                    late[h] = (tok >= min_keys ? 0x8000u : 0u) | (tok + 1 >= min_keys ? 0x80000000u : 0u);
                }
            }
            const auto values = [&](int m, uint32_t v[4]) {         // v: rows r8, r8 + 8 of keys 0-7, then of 8-15
                if (kEdge) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] &= keep[e >> 1];
                    // A weight of zero does not keep a NaN out of a product, so what is not finite leaves
                    // the operand here, and the columns that attend it get their NaN in the sum itself.
                    uint32_t lost[4], any = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) any |= lost[e] = not_finite<kFp8>(v[e]) & late[e >> 1];
                    if (__any_sync(~0u, any)) {
#pragma unroll
                        for (int d = 0; d < 2; ++d) {              // row r8, then r8 + 8
                            int from = INT_MAX;                    // first such token
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int tok = t0 + 8 * h + 2 * j4;
                                const uint32_t x = lost[2 * h + d];
                                if (x >> 31) from = min(from, tok + 1);
                                if (x & 0x8000u) from = min(from, tok);
                                v[2 * h + d] &= ~((x >> 15) * 0xffffu);
                            }
                            from = min(from, __shfl_xor_sync(~0u, from, 1));
                            from = min(from, __shfl_xor_sync(~0u, from, 2));
#pragma unroll
                            for (int t = 0; t < L; ++t)
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    if (from < keys_of(t, c)) o[t][m][2 * d + c] = __int_as_float(0x7fffffff);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < L; ++t) mma16<kFp8>(o[t][m], v, p[t][0], p[t][1]);
            };
#pragma unroll
            for (int s = 0; s < (kFp8 ? 4 : 8); ++s) {
                uint32_t w[4];
                load4_transposed(w, (chunk + v_lane) ^ (s << 5));
                if (kFp8) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t lo = __byte_perm(w[2 * u], 0, 0x3120), hi = __byte_perm(w[2 * u + 1], 0, 0x3120);
                        uint32_t v[4] = {halves_of(lo), halves_of(lo >> 16), halves_of(hi), halves_of(hi >> 16)};
                        values(2 * s + u, v);
                    }
                } else {
                    values(s, w);
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
        const float v_scale = kFp8 ? a.v_scale[kv] : 1.f;
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
                for (int m = 0; m < 8; ++m) {
                    float *to = mine_o + col * kOutStride + 16 * m + (kFp8 ? 2 * r8 : r8);
                    to[0] = o[t][m][c] * v_scale;
                    to[kFp8 ? 1 : 8] = o[t][m][c + 2] * v_scale;
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
            sc.open[blockIdx.x] = Open{min(b, blocks - 1) - (int)blockIdx.x + 1, q.row0, q.rows, kv, tile};
        }
        __syncthreads();
        at = item0 = next;
        ++tile;
    }
}

// Short caches are not worth cutting: an item stays with one block, and the second launch
// falls away.
bool whole_items(const PAttn &a) { return (long long)a.max_pages * (a.c.page_size / kChunk) <= kWholeChunks; }

// Columns up to which a request is worked on by columns, and not by tiles of 256 rows.  us by
// columns / tiles, 32 requests up to 8192 (32/8 heads): 20 columns bf16 100 / 109, e4m3 98 / 112; 32
// 105 / 109, 122 / 112; 64 (32/4 heads) 86 / 66, 152 / 73.  Short caches, which are not cut: 4 of 300
// tokens with 128 columns 13 / 17.
int most_columns(const PAttn &a) { return whole_items(a) ? 128 : a.k_scale ? 24 : 32; }
bool with_tiles(const PAttn &a) { return a.g <= kBlock && (long long)a.max_q * a.g > most_columns(a); }
// Whether requests of up to 8 columns are left to the columns where others go to tiles: a launch
// more, and an e4m3 cache's values that are not converted for a row or two, against tiles that hold
// all requests at once.  us by both / by tiles alone, 64 requests of 4096 to 8192 (64/8 heads), q rows
// in a part of them and 1 in the others: bf16 q 10 in 50% 288 / 281, 10 in 2% 276 / 278; 32/4 heads
// 155 / 150 and 164 / 151; but 128 requests to 4096, 64 in 5% 293 / 327, 256 in 1% 286 / 328.  e4m3 q 10
// in 2% 185 / 289, in 50% 248 / 294, in all 303 / 296.  12 to 32 heads a KV head: bf16 203 / 191 and
// 181 / 161, e4m3 164 / 156, 177 / 172 and (2% of 16 rows) 157 / 171.
// A request of more than 8 columns would read its keys once for every 8 of them: drafts of 1 to 5 rows,
// bf16 588 by such columns, 276 by tiles.
constexpr int kBeside = 8;
bool with_columns(const PAttn &a) {
    if (!with_tiles(a)) return true;
    if (!a.cu || a.g > kBeside) return false;
    return a.k_scale ? a.total_q != (long long)a.batch * a.max_q : (long long)a.max_q * a.g > kBlock;
}

// Columns of a tile.  Where every request has max_q rows, as many as it has, up to 32;
// where the rows differ, what most of them fill, by the mean that the host knows.
int tile_columns(const PAttn &a) {
    if (with_tiles(a)) return kBeside;
    const long long cols = (long long)a.max_q * a.g, all = (long long)a.total_q * a.g;
    const bool ragged = a.cu && a.total_q != (long long)a.batch * a.max_q;
    if (cols <= 8 || (ragged && all <= 8ll * a.batch)) return 8;
    return cols <= 16 || (ragged && all <= 16ll * a.batch) ? 16 : 32;
}

template <bool kFp8>
int per_sm_of(int cols) {
    return cols == 8 ? blocks_per_sm<kFp8, 1>() : cols == 16 ? blocks_per_sm<kFp8, 2>() : blocks_per_sm<kFp8, 4>();
}

int blocks_of(const PAttn &a) {
    const int cols = tile_columns(a);
    const int most = kSm * (a.k_scale ? per_sm_of<true>(cols) : per_sm_of<false>(cols));
    // no more than the longest lengths that the table can hold would use
    const long long rows = a.cu ? a.total_q : (long long)a.batch * a.max_q;
    const double items = (double)a.c.h_kv * (rows * a.g / cols + a.batch);
    if (a.whole) return items < (double)most ? (int)items : most;
    const double chunks = items * ((double)a.max_pages * (a.c.page_size / kChunk) + 40);
    return chunks < (double)most * kMinChunks ? (int)(chunks / kMinChunks) + 1 : most;
}

template <bool kFp8, int NT>
cudaError_t launch(const PAttn &a, const Scratch &sc, int blocks, cudaStream_t st) {
    constexpr int ring = stages<kFp8, NT>() * chunk_bytes<kFp8>(), smem = kWarps * ring + 256;
    static_assert(ring >= 8 * NT * kOutStride * 4, "a warp's result fits its ring");
    static_assert(ring % 256 == 0, "rings stay aligned");
    static std::atomic<unsigned long long> told{0};
    const cudaError_t e = launch_large(told, columns_kernel<kFp8, NT>, blocks, kThreads, smem, st, a, sc);
    if (e != cudaSuccess) return e;
    if (a.whole) return cudaSuccess;
    return launch_chained(join_kernel<NT, most_blocks<kFp8>(), PAttn>, blocks < 2 * kSm ? blocks : 2 * kSm, kJoinWarps * 32, 0,
                          st, a, sc, blocks);
}

template <bool kFp8>
cudaError_t launch_columns(const PAttn &a, const Scratch &sc, int cols, int blocks, cudaStream_t st) {
    switch (cols) {
        case 8: return launch<kFp8, 1>(a, sc, blocks, st);
        case 16: return launch<kFp8, 2>(a, sc, blocks, st);
        default: return launch<kFp8, 4>(a, sc, blocks, st);
    }
}

}  // namespace

size_t cache_attn_scratch_bytes(const PAttn &args) {
    PAttn a = args;
    a.whole = whole_items(a);
    const size_t n = blocks_of(a), cols = tile_columns(a);
    const size_t columns =
        align256(n * sizeof(Open)) + align256(n * 2 * cols * sizeof(float2)) + n * 2 * cols * kHeadDim * sizeof(float);
    const size_t tiles = with_tiles(a) ? cache_tiles_scratch_bytes(a) : 0;       // one after the other in the same memory
    return with_columns(a) && columns > tiles ? columns : tiles;
}

cudaError_t launch_cache_attn(const PAttn &args, void *scratch, unsigned long long limit_ns, cudaStream_t st) {
    PAttn a = args;
    a.whole = whole_items(a);
    a.most_columns = with_tiles(a) ? (with_columns(a) ? kBeside : 0) : INT_MAX;
    if (with_columns(a)) {
        const size_t n = blocks_of(a), cols = tile_columns(a);
        char *p = static_cast<char *>(scratch);
        Scratch sc;
        sc.open = reinterpret_cast<Open *>(p);
        p += align256(n * sizeof(Open));
        sc.ml = reinterpret_cast<float2 *>(p);
        p += align256(n * 2 * cols * sizeof(float2));
        sc.o = reinterpret_cast<float *>(p);
        const cudaError_t e = a.k_scale ? launch_columns<true>(a, sc, (int)cols, (int)n, st)
                                        : launch_columns<false>(a, sc, (int)cols, (int)n, st);
        if (e != cudaSuccess) return e;
    }
    return with_tiles(a) ? launch_cache_tiles(a, scratch, limit_ns, st) : cudaSuccess;
}

}  // namespace fp
