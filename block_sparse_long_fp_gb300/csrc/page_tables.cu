// fp_page_tables: block tables, lengths and slot maps of one step.
//
// A step is a scan over the batch (tokens and pages of each request) and then
// one independent look-up per token.  Every thread block scans the whole batch
// for itself -- 8 bytes a request from L2 -- so that one launch does it all;
// the tokens and the new table entries are dealt over the blocks.  Bound by that
// chain's latency: 64 requests of one token 3.3 us, 128 requests with 524288
// tokens (4 MB of maps) 7.4 us.
#include "qcache.cuh"

namespace fp {
namespace {

struct Plan {
    int cu;        // first row
    int old;       // cached tokens; for a refused request, -1
    int off;       // first of its entries of free_pages
    int len;       // new tokens
};

// Exclusive scan of a pair over the block; returns the totals in *sum.
__device__ __forceinline__ longlong2 block_scan(longlong2 v, longlong2 *sum, longlong2 *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    longlong2 x = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const long long a = __shfl_up_sync(~0u, x.x, d), b = __shfl_up_sync(~0u, x.y, d);
        if (lane >= d) x.x += a, x.y += b;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    longlong2 before = make_longlong2(0, 0), all = make_longlong2(0, 0);
    for (int w = 0; w < warps; ++w) {
        const longlong2 s = warp_sums[w];
        if (w < warp) before.x += s.x, before.y += s.y;
        all.x += s.x, all.y += s.y;
    }
    __syncthreads();
    *sum = all;
    return make_longlong2(before.x + x.x - v.x, before.y + x.y - v.y);
}

// Most threads of a block, which a step in place takes.  Left to itself the kernel of eight
// tokens a thread takes 66 registers, and an SM's 65536 do not hold 1024 threads of it.
template <int kTokens>
constexpr int most_threads() { return kTokens == 1 ? 1024 : 512; }

// kTokens: consecutive tokens per thread.
template <int kTokens>
__global__ void __launch_bounds__(most_threads<kTokens>()) tables_kernel(fp_tables t, int shift, int *status) {
    extern __shared__ Plan plan[];               // [batch]
    __shared__ longlong2 warp_sums[32];
    __shared__ long long taken;
    after_previous();
    const int nthr = blockDim.x;
    const bool first = blockIdx.x == 0;
    // shift: log2 of page_size, or -1 where it is no power of two
    const auto page_of = [&](int pos) { return shift >= 0 ? pos >> shift : pos / t.page_size; };
    const auto pages = [&](long long tokens) {
        tokens += t.page_size - 1;
        return shift >= 0 ? tokens >> shift : tokens / t.page_size;
    };
    const int head = t.free_head ? *t.free_head : 0;
    const long long avail = head < 0 ? 0 : (long long)t.num_free - head;
    if (threadIdx.x == 0) taken = 0;
    longlong2 carry = make_longlong2(0, 0);
    bool refused = false;
    for (int base = 0; base < t.batch; base += nthr) {
        const int r = base + threadIdx.x;
        long long old = 0, add = 0, need = 0;
        bool ok = true;
        if (r < t.batch) {
            old = t.seqlens[r];
            add = t.new_lens[r];
            const long long all = old >= 0 && add >= 0 && old + add <= 0x7fffffffll ? pages(old + add) : -1;
            ok = all >= 0 && all <= t.max_pages_per_seq;
            need = ok ? all - pages(old) : 0;
            if (add < 0) add = 0;
        }
        longlong2 sum;
        const longlong2 at = block_scan(make_longlong2(add, need), &sum, warp_sums);
        if (r < t.batch) {
            const long long cu = carry.x + at.x, off = carry.y + at.y;
            ok = ok && (need == 0 || off + need <= avail) && (add == 0 || cu + add <= t.capacity);
            if (ok && need) atomicMax((unsigned long long *)&taken, (unsigned long long)(off + need));
            refused |= !ok;
            Plan p;
            p.cu = (int)min(cu, 0x7fffffffll);
            p.old = ok ? (int)old : -1;
            p.off = (int)min(off, 0x7fffffffll);
            p.len = (int)add;
            plan[r] = p;
            if (first) {
                t.cu_seqlens_q[r] = p.cu;
                t.seqlens_k[r] = (int)(ok ? old + add : old);
            }
        }
        carry.x += sum.x;
        carry.y += sum.y;
    }
    __syncthreads();
    if (first) {
        if (threadIdx.x == 0) {
            t.cu_seqlens_q[t.batch] = (int)min(carry.x, 0x7fffffffll);
            *t.free_next = head + (int)taken;
        }
        if (refused || head < 0 || head > t.num_free) set_status(status, FP_ERR_DEVICE_BOUNDS);
    }
    // new table entries: entry n of the scan belongs to the last request whose first is at or before it
    const int gthreads = gridDim.x * nthr, gthread = blockIdx.x * nthr + threadIdx.x;
    const long long entries = min(carry.y, avail);
    for (long long n = gthread; n < entries; n += gthreads) {
        int lo = 0, hi = t.batch - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (plan[mid].off <= n) lo = mid; else hi = mid - 1;
        }
        const Plan p = plan[lo];
        if (p.old >= 0)
            t.block_table[(long long)lo * t.max_pages_per_seq + pages(p.old) + n - p.off] = t.free_pages[head + n];
    }
    // tokens
    for (long long i0 = (long long)gthread * kTokens; i0 < t.capacity; i0 += (long long)gthreads * kTokens) {
        int lo = 0, hi = t.batch - 1;            // the last request that starts at or before i0
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (plan[mid].cu <= i0) lo = mid; else hi = mid - 1;
        }
        int r = lo, pos[kTokens], slot[kTokens];
        const int *from[kTokens];                // where the token's page id is
        Plan p = plan[r];
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            const long long i = i0 + j;
            while (i - p.cu >= p.len && r + 1 < t.batch) p = plan[++r];
            const long long local = i - p.cu;
            const bool live = local < p.len && p.old >= 0;
            pos[j] = live ? p.old + (int)local : 0;
            const int pg = page_of(pos[j]), used = live ? (int)pages(p.old) : 0;
            from[j] = !live ? nullptr
                            : pg < used ? t.block_table + (long long)r * t.max_pages_per_seq + pg
                                        : t.free_pages + head + p.off + pg - used;
        }
#pragma unroll
        for (int j = 0; j < kTokens; ++j) slot[j] = from[j] ? *from[j] : -1;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            const bool in = slot[j] >= 0 && slot[j] < t.num_pages;
            bad |= from[j] && !in;
            slot[j] = from[j] && in ? slot[j] * t.page_size + pos[j] - page_of(pos[j]) * t.page_size : -1;
        }
        if (bad) set_status(status, FP_ERR_DEVICE_BOUNDS);
        if (kTokens % 4 == 0 && i0 + kTokens <= t.capacity) {
#pragma unroll
            for (int j = 0; j + 3 < kTokens; j += 4) {
                *reinterpret_cast<int4 *>(t.positions + i0 + j) = make_int4(pos[j], pos[j + 1], pos[j + 2], pos[j + 3]);
                *reinterpret_cast<int4 *>(t.slots + i0 + j) = make_int4(slot[j], slot[j + 1], slot[j + 2], slot[j + 3]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kTokens; ++j)
                if (i0 + j < t.capacity) {
                    t.positions[i0 + j] = pos[j];
                    t.slots[i0 + j] = slot[j];
                }
        }
    }
}

}  // namespace

cudaError_t launch_page_tables(const fp_tables &t, int *status, cudaStream_t st) {
    // Advancing lengths or the free list in place needs every read before the
    // first write: one block, whose scan ends in a barrier, does that.  64 tokens
    // 7.5 us, 70400 68 us, 524288 327 us; with arrays apart, measured alike, 4.8, 5.1, 7.7 us.
    const bool in_place = t.seqlens_k == t.seqlens || t.free_next == t.free_head;
    // One token per thread while that fills the GPU no more than twice: the call is
    // bound by the latency of the look-ups (a decode step of 64 requests: 3.3 us, and
    // 25 us with 8 tokens per thread one after the other).  Longer ones take 8, whose
    // look-ups go out together: one scan of the batch for 2048 tokens.
    const int tokens = t.capacity <= 2 * 152 * 256 ? 1 : 8;
    const int threads = !in_place ? 256 : tokens == 1 ? most_threads<1>() : most_threads<8>();
    const long long per_block = (long long)threads * tokens;
    long long grid = in_place ? 1 : (t.capacity + per_block - 1) / per_block;
    if (grid > 2 * 152) grid = 2 * 152;
    const size_t smem = (size_t)t.batch * sizeof(Plan);
    const auto kernel = tokens == 1 ? tables_kernel<1> : tables_kernel<8>;
    if (smem > 47 * 1024) {      // the limit without leave is 48 KB, with the static part of 528 bytes
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   FP_TABLES_MAX_BATCH * (int)sizeof(Plan));
        if (e != cudaSuccess) return e;
    }
    const int shift = (t.page_size & (t.page_size - 1)) == 0 ? __builtin_ctz(t.page_size) : -1;
    return launch_chained(kernel, (unsigned)grid, threads, smem, st, t, shift, status);
}

}  // namespace fp
