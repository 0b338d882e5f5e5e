// fp_qcache_write and fp_qcache_read: rows of bf16 or e4m3 to the 4-bit cache
// and back.
//
// Both are bound by memory where there are many rows: per (token, head) 512 bytes of bf16
// on one side and 128 + 1024 / G bytes of cache on the other.  65536 tokens of 8 heads
// (groups of 32) are written in 66 us, 5.3 TB/s, 0.78 of the measured copy rate (three
// quarters of the issue slots go to the quantisation; from e4m3 in 71), and 131072 of 4 heads
// read in 62 us, 5.7 TB/s, 0.84 (65536 of 8 heads to e4m3 in 62, which is arithmetic).  Few
// rows are bound by the latency of one dependent chain (slot, row, extremes, store), 2 us, and
// take a warp per (row, kv head): four dims per lane, so that a group of G dims is G / 4
// neighbouring lanes and its extremes take log2(G / 4) shuffles.
#include <type_traits>

#include "qcache.cuh"

namespace fp {
namespace {

constexpr int kWarps = 4;
// (row, head) pairs from which on a warp takes 16 rows of a head.  Microseconds with a warp a
// pair / with 16 rows a warp, for 8 heads in groups of 32, at 4096, 8192, 16384, 32768 pairs:
//   slots in order:  bf16 written  3.2 / 3.8   4.4 / 4.0   7.5 / 4.7  13.3 /  6.4
//                    bf16 read     2.3 / 2.7   3.1 / 3.0   4.7 / 3.8   8.3 /  5.3
//                    e4m3 written  3.2 / 3.3   4.8 / 3.6   8.0 / 4.4  14.5 /  6.0
//                    e4m3 read     3.4 / 3.2   4.6 / 3.5   7.4 / 4.3  12.5 /  5.8
//   a page each:     bf16 written  3.2 / 5.0   4.5 / 5.6   7.7 / 7.3  15.4 / 15.2
//                    bf16 read     2.3 / 4.6   3.1 / 4.9   5.7 / 8.0  11.5 / 14.6
//                    e4m3 written  3.2 / 4.1   4.8 / 4.4   8.0 / 5.5  15.8 / 11.8
//                    e4m3 read     3.4 / 5.2   4.7 / 5.5   7.6 / 7.7  13.5 / 14.5
// The host does not know the slots: the number is where single tokens of many requests stop
// losing by it when written, above where prompts begin to gain.
constexpr long long kManyRows = 16384;

__device__ __forceinline__ void load4(const void *base, long long elem, const float *scale, int head, float x[4]) {
    if (scale) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const unsigned char *>(base) + elem);
        const float s = scale[head];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_fp8_e4m3 c;
            c.__x = (__nv_fp8_storage_t)((w >> (8 * i)) & 0xff);
            x[i] = (float)c * s;
        }
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(base) + elem);
        x[0] = __uint_as_float(w.x << 16);
        x[1] = __uint_as_float(w.x & 0xffff0000u);
        x[2] = __uint_as_float(w.y << 16);
        x[3] = __uint_as_float(w.y & 0xffff0000u);
    }
}

// The four codes of this lane in the low 16 bits, and its group's step and minimum.
template <int GROUPS>
__device__ __forceinline__ uint32_t quantise(float x[4], __half *step, __half *low) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        nan |= x[i] != x[i];
        x[i] = fminf(fmaxf(x[i], -65504.f), 65504.f);
    }
    float mn = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
    float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    unsigned bad = nan;
#pragma unroll
    for (int d = 1; d < 32 / GROUPS; d *= 2) {
        mn = fminf(mn, __shfl_xor_sync(~0u, mn, d));
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
        bad |= __shfl_xor_sync(~0u, bad, d);
    }
    const __half m = bad ? __ushort_as_half(0x7e00) : __float2half_rn(mn);
    const float mf = __half2float(m);
    const __half s = bad ? __ushort_as_half(0) : __float2half_rn(fminf(fmaxf((mx - mf) / 15.f, 0.f), 65504.f));
    const float sf = __half2float(s);
    const float inv = sf > 0.f ? 1.f / sf : 0.f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float c = fminf(fmaxf(rintf((x[i] - mf) * inv), 0.f), 15.f);
        w |= (uint32_t)c << (4 * i);
    }
    *step = s;
    *low = m;
    return w;
}

template <int GROUPS>
__global__ void __launch_bounds__(kWarps * 32) write_kernel(QCache c, QRows r, int *status) {
    after_previous();
    const long long unit = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
    if (unit >= (long long)r.rows * c.h_kv) return;
    const int row = (int)(unit / c.h_kv), head = (int)(unit - (long long)row * c.h_kv), l = threadIdx.x & 31;
    const int slot = r.slots[row];
    if (slot < 0 || slot >= c.num_pages * c.page_size) {
        if (slot != -1 && l == 0) set_status(status, FP_ERR_DEVICE_BOUNDS);
        return;
    }
    const long long at = row * r.stride_tok + head * r.stride_head + 4 * l;
    float k[4], v[4];
    load4(r.k, at, r.k_scale, head, k);
    load4(r.v, at, r.v_scale, head, v);
    unsigned char *chunk = qcache_chunk(c, slot, head);
    const int t = slot % kChunk, lane_group = l * GROUPS / 32;
    __half s, m;
    *reinterpret_cast<uint16_t *>(chunk + k_code_off(t, l)) = (uint16_t)quantise<GROUPS>(k, &s, &m);
    if (l % (32 / GROUPS) == 0) {
        __half *p = reinterpret_cast<__half *>(chunk + k_step_off(t, lane_group, GROUPS));
        p[0] = s;
        p[16 * GROUPS] = m;
    }
    *reinterpret_cast<uint16_t *>(chunk + v_code_off(t, l)) = (uint16_t)quantise<GROUPS>(v, &s, &m);
    if (l % (32 / GROUPS) == 0) {
        __half *p = reinterpret_cast<__half *>(chunk + v_step_off(t, lane_group, GROUPS));
        p[0] = s;
        p[16 * GROUPS] = m;
    }
}

// s * c is exact in fp32 (11 + 4 bits), so the fused product and sum rounds once.
__device__ __forceinline__ void dequantise(uint32_t w, const __half *p, int groups, float x[4]) {
    const float s = __half2float(p[0]), m = __half2float(p[16 * groups]);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = fmaf(s, (float)((w >> (4 * i)) & 15u), m);
}

__device__ __forceinline__ void store4(void *base, long long elem, const float *scale, int head, const float x[4]) {
    if (scale) {
        const float s = scale[head];
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w |= (uint32_t)__nv_cvt_float_to_fp8(x[i] / s, __NV_SATFINITE, __NV_E4M3) << (8 * i);
        *reinterpret_cast<uint32_t *>(static_cast<unsigned char *>(base) + elem) = w;
    } else {
        __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(base) + elem) =
            make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
    }
}

template <int GROUPS>
__global__ void __launch_bounds__(kWarps * 32) read_kernel(QCache c, QRows r, int *status) {
    after_previous();
    const long long unit = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
    if (unit >= (long long)r.rows * c.h_kv) return;
    const int row = (int)(unit / c.h_kv), head = (int)(unit - (long long)row * c.h_kv), l = threadIdx.x & 31;
    const int slot = r.slots[row], to = r.out_slots ? r.out_slots[row] : row;
    if (slot < 0 || slot >= c.num_pages * c.page_size || to < 0 || to >= r.out_rows) {
        if (slot != -1 && to != -1 && l == 0) set_status(status, FP_ERR_DEVICE_BOUNDS);
        return;
    }
    const unsigned char *chunk = qcache_chunk(c, slot, head);
    const int t = slot % kChunk, lane_group = l * GROUPS / 32;
    const long long at = to * r.stride_tok + head * r.stride_head + 4 * l;
    float x[4];
    dequantise(*reinterpret_cast<const uint16_t *>(chunk + k_code_off(t, l)),
               reinterpret_cast<const __half *>(chunk + k_step_off(t, lane_group, GROUPS)), GROUPS, x);
    store4(const_cast<void *>(r.k), at, r.k_scale, head, x);
    dequantise(*reinterpret_cast<const uint16_t *>(chunk + v_code_off(t, l)),
               reinterpret_cast<const __half *>(chunk + v_step_off(t, lane_group, GROUPS)), GROUPS, x);
    store4(const_cast<void *>(r.v), at, r.v_scale, head, x);
}

// -- many rows: a warp takes 16 rows of a head at a time ------------------------------
//
// Tokens share a chunk's bytes in an order that only whole chunks write well (a V
// token is eight pieces of 8 bytes), so a warp builds the chunk's image in shared
// memory, 16 dims per lane, and moves it in 16-byte pieces when its 16 rows are one
// chunk; other rows go piece by piece.  For that the rows are cut where their slots
// begin a chunk, wherever that falls: a run is a stretch of consecutive slots inside
// a chunk, and window w owns the runs that start in rows 16 w .. 16 w + 15.

struct Owned {
    int first, end;        // rows
    int slot;              // of row 16 w + lane (-1 behind the last row)
};

__device__ __forceinline__ Owned owned_rows(const int *slots, int rows, int w) {
    const int lane = threadIdx.x & 31, row = w * kChunk + lane;
    Owned o;
    o.slot = row < rows ? slots[row] : -1;
    int before = __shfl_up_sync(~0u, o.slot, 1);
    if (lane == 0) before = row > 0 ? slots[row - 1] : -2;
    const unsigned starts =
        __ballot_sync(~0u, row < rows && (o.slot < 0 || o.slot % kChunk == 0 || o.slot != before + 1));
    const unsigned own = starts & 0xffffu, next = starts & 0xffff0000u;
    // a run is at most 16 rows, so the next one starts, or the rows end, within these 32
    o.first = own ? w * kChunk + __ffs(own) - 1 : 0;
    o.end = own ? (next ? w * kChunk + __ffs(next) - 1 : min(rows, w * kChunk + 32)) : 0;
    return o;
}

// A warp takes either the keys (V = false) or the values of its rows: a half chunk, its
// codes and its f16 arrays, which lie at these offsets in the chunk and one behind the
// other in the image.
template <int GROUPS, bool V>
struct Half {
    static constexpr int kMeta = 64 * GROUPS, kImage = kCodeBytes + kMeta;
    static constexpr int kCodesAt = V ? kCodeBytes : 0, kMetaAt = 2 * kCodeBytes + (V ? kMeta : 0);
    // the 2 bytes of dims 4 l .. 4 l + 3 of token t, and the step of its group g, in the image
    static __device__ __forceinline__ int code(int t, int l) { return V ? v_code_off(t, l) - kCodesAt : k_code_off(t, l); }
    static __device__ __forceinline__ int step(int t, int g) {
        return kCodeBytes - kMetaAt + (V ? v_step_off(t, g, GROUPS) : k_step_off(t, g, GROUPS));
    }
    // from an offset in the image to the one in the chunk
    static __device__ __forceinline__ int in_chunk(int at) { return at + (at < kCodeBytes ? kCodesAt : kMetaAt - kCodeBytes); }
};

// Sixteen tokens between their chunks and an image of 16 tokens, all at once: a token's
// keys are 4 pieces of 16 bytes and 2 (steps, minima) of 2 GROUPS, its values 8 of 8 and
// 2 GROUPS of 2.  `mine` is the chunk of token lane & 15, its place in the chunk in the
// low four bits, 0 for none.
template <typename H, typename T, int N, bool TO_CHUNKS, typename F>
__device__ __forceinline__ void move_pieces(unsigned long long mine, unsigned char *img, F piece) {
    unsigned char *at[N];
    int in[N];
    T x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {                // piece(i, t): the token, then its offset as token t of a chunk
        const int t = piece(i, -1);
        const unsigned long long chunk = __shfl_sync(~0u, mine, t);
        at[i] = chunk ? reinterpret_cast<unsigned char *>(chunk & ~15ull) + H::in_chunk(piece(i, (int)(chunk & 15)))
                      : nullptr;
        in[i] = piece(i, t);
        if (at[i]) x[i] = *reinterpret_cast<const T *>(TO_CHUNKS ? img + in[i] : at[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (at[i]) *reinterpret_cast<T *>(TO_CHUNKS ? at[i] : img + in[i]) = x[i];
}

template <int GROUPS, bool V, bool TO_CHUNKS>
__device__ __forceinline__ void move_tokens(unsigned long long mine, unsigned char *img) {
    using H = Half<GROUPS, V>;
    using Meta = typename std::conditional<GROUPS == 4, uint2, typename std::conditional<GROUPS == 2, uint32_t, uint16_t>::type>::type;
    const int l = threadIdx.x & 31;
    if (V) {
        move_pieces<H, uint2, 4, TO_CHUNKS>(mine, img, [&](int i, int t) { return t < 0 ? (i * 32 + l) / 8 : H::code(t, l % 8); });
        move_pieces<H, uint16_t, GROUPS, TO_CHUNKS>(mine, img, [&](int i, int t) {
            const int e = (i * 32 + l) % (2 * GROUPS);
            return t < 0 ? (i * 32 + l) / (2 * GROUPS) : H::step(t, e % GROUPS) + e / GROUPS * 32 * GROUPS;
        });
    } else {
        move_pieces<H, uint4, 2, TO_CHUNKS>(mine, img, [&](int i, int t) { return t < 0 ? (i * 32 + l) / 4 : t * 64 + l % 4 * 16; });
        move_pieces<H, Meta, 1, TO_CHUNKS>(mine, img,
                                           [&](int, int t) { return t < 0 ? l / 2 : H::step(t, 0) + l % 2 * 32 * GROUPS; });
    }
}

// Sixteen dims of a row, as they lie in memory.
template <bool FP8>
struct Raw {
    uint4 w[FP8 ? 1 : 2];
};
template <bool FP8>
__device__ __forceinline__ Raw<FP8> load16(const void *base, long long elem, bool live) {
    Raw<FP8> r;
    r.w[0] = r.w[FP8 ? 0 : 1] = make_uint4(0, 0, 0, 0);
    if (!live) return r;
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(base) + elem * (FP8 ? 1 : 2));
    r.w[0] = p[0];
    if (!FP8) r.w[FP8 ? 0 : 1] = p[1];
    return r;
}
template <bool FP8>
__device__ __forceinline__ void unpack16(const Raw<FP8> &r, float scale, float x[16]) {
    if (FP8) {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __half2_raw h =
                __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            x[2 * i] = f.x * scale;
            x[2 * i + 1] = f.y * scale;
        }
    } else {
        const uint4 a = r.w[0], b = r.w[FP8 ? 0 : 1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

// The least and greatest of three, NaN if one is.
__device__ __forceinline__ float min_nan(float a, float b, float c) {
    float y;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// d / 15 and 1 / s as correctly rounded quotients need them: a quotient by the rounded
// reciprocal, corrected by its fused remainder (Markstein 1990), and a Newton step on the
// approximate reciprocal.  Equal to the division: the first for all 2^24 d of two binades
// (the others scale), the second in every code of ties by each fp16 s, which the tests take.
__device__ __forceinline__ float fifteenth(float d) {
    constexpr float kR = 1.f / 15.f;
    const float q = __fmul_rn(d, kR);
    return fmaf(fmaf(-15.f, q, d), kR, q);
}
__device__ __forceinline__ float reciprocal(float s) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
    return fmaf(fmaf(-s, y, 1.f), y, y);
}

// Eight codes, the first in the low bits, of eight values: (x - minimum) / step to the
// nearest, by adding 1.5 2^23, which leaves the code in the sum's low bits.  Products and
// sums stay apart: a fused one would round a tie that the product's rounding makes
// otherwise.  The assembler joins a packed product and the sum behind it into one rounding
// for all that both say .rn, and a fused product with a zero that it can see is a product
// to it: `zeros`, a pair of -0, comes from where it cannot.  Without `clamp` the codes are
// known to be in 0 .. 15.
__device__ __forceinline__ uint32_t codes8(const float_pair x[4], float low, float inv, float_pair zeros,
                                           bool clamp) {
    const float_pair minus = pair(-low, -low), by = pair(inv, inv), magic = pair(12582912.f, 12582912.f);
    uint32_t w = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        float_pair y = fma2(add2(x[i], minus), by, zeros);
        if (clamp) {
            const float2 v = unpair(y);
            y = pair(fminf(fmaxf(v.x, 0.f), 15.f), fminf(fmaxf(v.y, 0.f), 15.f));
        }
        const float2 v = unpair(add2(y, magic));
        w = w * 256 + __float_as_uint(v.y) * 16 + __float_as_uint(v.x);
    }
    return w - 0x4b400000u * 0x11111111u;        // the magic's own bits, eight times
}

// Sixteen codes of a lane, their group's step and minimum.  The group's least and greatest
// value say whether any of it needs the clamps, which are a path of their own.
template <int GROUPS, bool FP8>
__device__ __forceinline__ uint2 quantise16(const Raw<FP8> &raw, float scale, float_pair zeros, __half *step,
                                            __half *low) {
    float mn, mx;
    if (FP8) {
        float x[16];
        unpack16<FP8>(raw, scale, x);
        mn = mx = x[0];
#pragma unroll
        for (int i = 1; i < 16; i += 2) {
            const float b = x[i], c = x[i + 1 < 16 ? i + 1 : i];
            mn = min_nan(mn, b, c);
            mx = max_nan(mx, b, c);
        }
    } else {                                     // bf16 two at a time, as they lie
        const uint4 a = raw.w[0], b = raw.w[FP8 ? 0 : 1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        __nv_bfloat162 lo = *reinterpret_cast<const __nv_bfloat162 *>(&w[0]), hi = lo;
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            lo = __hmin2_nan(lo, *reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
            hi = __hmax2_nan(hi, *reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
        }
        const float2 l = __bfloat1622float2(lo), h = __bfloat1622float2(hi);
        mn = min_nan(l.x, l.y, l.y);
        mx = max_nan(h.x, h.y, h.y);
    }
#pragma unroll
    for (int d = 1; d < 8 / GROUPS; d *= 2) {
        mn = min_nan(mn, mn, __shfl_xor_sync(~0u, mn, d));
        mx = max_nan(mx, mx, __shfl_xor_sync(~0u, mx, d));
    }
    const bool far = !(mn >= -65504.f && mx <= 65504.f);
    if (far) {
        if (mn != mn) {                          // a NaN in the group
            *step = __ushort_as_half(0);
            *low = __ushort_as_half(0x7e00);
            return make_uint2(0, 0);
        }
        mn = fminf(fmaxf(mn, -65504.f), 65504.f);
        mx = fminf(fmaxf(mx, -65504.f), 65504.f);
    }
    const __half m = __float2half_rn(mn);
    const float mf = __half2float(m);
    const __half s = __float2half_rn(fminf(fmaxf(fifteenth(__fsub_rn(mx, mf)), 0.f), 65504.f));
    const float sf = __half2float(s);
    const float inv = sf > 0.f ? reciprocal(sf) : 0.f;
    *step = s;
    *low = m;
    const bool clamp =
        far || __fmul_rn(__fsub_rn(mn, mf), inv) < -0.5f || __fmul_rn(__fsub_rn(mx, mf), inv) >= 15.5f;
    uint32_t code[2];
    if (clamp) {
        float x[16];
        unpack16<FP8>(raw, scale, x);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float_pair y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[i] = pair(fminf(fmaxf(x[8 * h + 2 * i], -65504.f), 65504.f),
                            fminf(fmaxf(x[8 * h + 2 * i + 1], -65504.f), 65504.f));
            code[h] = codes8(y, mf, inv, zeros, true);
        }
    } else {
        float x[16];
        unpack16<FP8>(raw, scale, x);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float_pair y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = pair(x[8 * h + 2 * i], x[8 * h + 2 * i + 1]);
            code[h] = codes8(y, mf, inv, zeros, false);
        }
    }
    return make_uint2(code[0], code[1]);
}

// The rows of a warp, 16 at a time: body(first row, rows, slot of row lane & 15, its
// chunk's address when the 16 are one whole chunk, else null).
template <typename F>
__device__ __forceinline__ void for_owned(const QCache &c, const QRows &r, int w, int head, F body) {
    const int lane = threadIdx.x & 31;
    const Owned own = owned_rows(r.slots, r.rows, w);
    for (int row0 = own.first; row0 < own.end; row0 += kChunk) {
        const int n = min(kChunk, own.end - row0);
        const int slot0 = __shfl_sync(~0u, own.slot, (row0 - w * kChunk) & 31);
        const int mine = __shfl_sync(~0u, own.slot, (row0 - w * kChunk + (lane & 15)) & 31);
        const bool whole = n == kChunk && slot0 % kChunk == 0 && __all_sync(~0u, mine == slot0 + (lane & 15)) &&
                           slot0 >= 0 && slot0 < c.num_pages * c.page_size;
        body(row0, n, mine, whole ? qcache_chunk(c, slot0, head) : nullptr);
    }
}

template <int GROUPS, bool FP8, bool V>
__device__ __forceinline__ void write_half(const QCache &c, const QRows &r, int w, int head, unsigned char *img, int *status) {
    using H = Half<GROUPS, V>;
    const int lane = threadIdx.x & 31, sub = lane / 8, part = lane % 8;      // row of four, 16 dims of the row
    const void *src = V ? r.v : r.k;
    const float zero = r.rows > 0 ? -0.f : 1.f;
    const float_pair zeros = pair(zero, zero);
    const float scale = FP8 ? (V ? r.v_scale : r.k_scale)[head] : 1.f;
    for_owned(c, r, w, head, [&](int row0, int n, int mine, unsigned char *chunk) {
        const auto load = [&](int i) {
            return load16<FP8>(src, (long long)(row0 + 4 * i + sub) * r.stride_tok + head * r.stride_head + 16 * part,
                               4 * i + sub < n);
        };
        // two steps a turn, as four unrolled do not fit the instruction cache (64K tokens of
        // bf16 written and read: 135 us, two 127, one 135), with the loads of e4m3, half as
        // many registers, two steps ahead (two 131 us, one 133)
        constexpr int kAhead = FP8 ? 2 : 1;
        Raw<FP8> raw[kAhead + 1];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) raw[i] = load(i);
#pragma unroll 2
        for (int i = 0; i < 4; ++i) {
            raw[kAhead] = load(i + kAhead);
            const int t = 4 * i + sub;
            __half s, m;
            const uint2 code = quantise16<GROUPS, FP8>(raw[0], scale, zeros, &s, &m);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) raw[k] = raw[k + 1];
            unsigned char *p = img + H::code(t, part * 4);
            if (V) {                             // dims 16 part .. + 15: four rows of four
                *reinterpret_cast<uint16_t *>(p) = (uint16_t)code.x;
                *reinterpret_cast<uint16_t *>(p + 64) = (uint16_t)(code.x >> 16);
                *reinterpret_cast<uint16_t *>(p + 128) = (uint16_t)code.y;
                *reinterpret_cast<uint16_t *>(p + 192) = (uint16_t)(code.y >> 16);
            } else {                             // two lanes of eight
                *reinterpret_cast<uint32_t *>(p) = code.x;
                *reinterpret_cast<uint32_t *>(p + 16) = code.y;
            }
            if (part % (8 / GROUPS) == 0) {
                __half *q = reinterpret_cast<__half *>(img + H::step(t, part * GROUPS / 8));
                q[0] = s;
                q[16 * GROUPS] = m;
            }
        }
        __syncwarp();
        if (chunk) {
#pragma unroll
            for (int b = lane * 16; b < H::kImage; b += 512)
                *reinterpret_cast<uint4 *>(chunk + H::in_chunk(b)) = *reinterpret_cast<const uint4 *>(img + b);
        } else {
            unsigned long long at = 0;
            if ((lane & 15) < n && mine != -1) {
                if (mine >= 0 && mine < c.num_pages * c.page_size)
                    at = (unsigned long long)qcache_chunk(c, mine, head) + mine % kChunk;
                else
                    set_status(status, FP_ERR_DEVICE_BOUNDS);
            }
            move_tokens<GROUPS, V, true>(at, img);
        }
        __syncwarp();
    });
}

template <int GROUPS, bool FP8, bool V>
__device__ __forceinline__ void read_half(const QCache &c, const QRows &r, int w, int head, unsigned char *img, int *status) {
    using H = Half<GROUPS, V>;
    const int lane = threadIdx.x & 31, sub = lane / 8, part = lane % 8;
    void *out = const_cast<void *>(V ? r.v : r.k);
    const float scale = FP8 ? (V ? r.v_scale : r.k_scale)[head] : 1.f;
    // a scale whose quotients and remainders could leave the normal numbers is divided by plainly
    const bool plain = !(fabsf(scale) >= 0x1p-60f && fabsf(scale) <= 0x1p60f);
    const float inverse = 1.f / scale, zero = r.rows > 0 ? -0.f : 1.f;
    const float_pair by = pair(inverse, inverse), minus = pair(-scale, -scale), zeros = pair(zero, zero);
    for_owned(c, r, w, head, [&](int row0, int n, int mine, unsigned char *chunk) {
        // target of row row0 + (lane & 15), -1 where nothing is to be written
        int to = -1;
        if ((lane & 15) < n && mine != -1) {
            const int row = row0 + (lane & 15), target = r.out_slots ? r.out_slots[row] : row;
            if (mine >= 0 && mine < c.num_pages * c.page_size && target >= 0 && target < r.out_rows)
                to = target;
            else if (target != -1)
                set_status(status, FP_ERR_DEVICE_BOUNDS);
        }
        if (chunk) {
            constexpr int kEach = (H::kImage + 511) / 512;
            uint4 x[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (i * 512 + lane * 16 < H::kImage)
                    x[i] = *reinterpret_cast<const uint4 *>(chunk + H::in_chunk(i * 512 + lane * 16));
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (i * 512 + lane * 16 < H::kImage) *reinterpret_cast<uint4 *>(img + i * 512 + lane * 16) = x[i];
        } else {
            move_tokens<GROUPS, V, false>(to >= 0 ? (unsigned long long)qcache_chunk(c, mine, head) + mine % kChunk : 0, img);
        }
        __syncwarp();
#pragma unroll 1                                 // registers and instruction cache again
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * i + sub, target = __shfl_sync(~0u, to, t);
            const unsigned char *p = img + H::code(t, part * 4);
            uint32_t code[2];
            if (V) {
                const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
                code[0] = q[0] | (uint32_t)q[32] << 16;
                code[1] = q[64] | (uint32_t)q[96] << 16;
            } else {
                code[0] = *reinterpret_cast<const uint32_t *>(p);
                code[1] = *reinterpret_cast<const uint32_t *>(p + 16);
            }
            const __half *q = reinterpret_cast<const __half *>(img + H::step(t, part * GROUPS / 8));
            const float s = __half2float(q[0]), m = __half2float(q[16 * GROUPS]);
            // Two codes at a time: a code 4 k bits up in the mantissa of 2^23 stands for 16^k
            // times itself, which the step's 16^-k takes back without a rounding.
            const float_pair steps[2] = {pair(s, s * 0x1p-4f), pair(s * 0x1p-8f, s * 0x1p-12f)};
            const float_pair less = pair(-8388608.f, -8388608.f), low = pair(m, m);
            float_pair x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t c4 = code[e / 4] >> (e & 2 ? 16 : 0), k = 8 * (e & 1);
                const float lo = __uint_as_float((c4 & 15u << k) | 0x4b000000u), hi = __uint_as_float((c4 & 240u << k) | 0x4b000000u);
                x[e] = fma2(steps[e & 1], add2(pair(lo, hi), less), low);
            }
            if (target < 0) continue;
            const long long at = target * r.stride_tok + head * r.stride_head + 16 * part;
            if (FP8) {
                if (plain) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 v = unpair(x[e]);
                        x[e] = pair(v.x / scale, v.y / scale);
                    }
                } else {                         // the same quotients by the rounded reciprocal (Markstein 1990)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float_pair f = fma2(x[e], by, zeros);
                        x[e] = fma2(fma2(f, minus, x[e]), by, f);
                    }
                }
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = __nv_cvt_float2_to_fp8x2(unpair(x[2 * e]), __NV_SATFINITE, __NV_E4M3) |
                           (uint32_t)__nv_cvt_float2_to_fp8x2(unpair(x[2 * e + 1]), __NV_SATFINITE, __NV_E4M3) << 16;
                *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(out) + at) = make_uint4(y[0], y[1], y[2], y[3]);
            } else {
                uint32_t y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 v = unpair(x[e]);
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
                    y[e] = *reinterpret_cast<const uint32_t *>(&h);
                }
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + at);
                dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
                dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
            }
        }
        __syncwarp();
    });
}

// Blocks an SM.  The kernels wait for memory and for their own arithmetic in turn, so that
// warps count for more than registers: the bf16 write spills 240 to 250 bytes a thread, the
// reads 90 to 140, the e4m3 write 40.  bf16 written at 8, 9, 10, 11, 13 blocks
// (64K tokens, and read back): 142, 134, 133, 127, 140 us; e4m3 at 8, 10, 11: 131, 129, 129 us,
// but 5003 tokens, which leave SMs unfilled: 12.6, 13.9, 14.1 us.  Read at 8, 9, 10, 11, 14
// blocks, 128K tokens to bf16: 66.7, 64.2, 64.0, 62.7, 73 us; 51327 tokens to e4m3: 49.4, 47.5,
// 47.7, 48.9, 58 us, 64K: 68, 66, 64, 63, 81 us.  (A warp that takes several heads in turn, the
// next one's loads ahead, has to spill for it: 63 us for 128K tokens, 133 us for 64K written.)
template <bool FP8, bool READ>
constexpr int rows_blocks() { return READ ? (FP8 ? 10 : 11) : FP8 ? 8 : 11; }

template <int GROUPS, bool FP8, bool READ>
__global__ void __launch_bounds__(kWarps * 32, (rows_blocks<FP8, READ>())) rows_kernel(QCache c, QRows r, int *status) {
    __shared__ __align__(16) unsigned char image[kWarps][Half<GROUPS, false>::kImage];
    after_previous();
    const long long unit = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
    const long long pair = unit / 2;
    const int w = (int)(pair / c.h_kv), head = (int)(pair - (long long)w * c.h_kv);
    if ((long long)w * kChunk >= r.rows) return;
    unsigned char *img = image[threadIdx.x / 32];
    if (READ) {
        if (unit & 1)
            read_half<GROUPS, FP8, true>(c, r, w, head, img, status);
        else
            read_half<GROUPS, FP8, false>(c, r, w, head, img, status);
    } else {
        if (unit & 1)
            write_half<GROUPS, FP8, true>(c, r, w, head, img, status);
        else
            write_half<GROUPS, FP8, false>(c, r, w, head, img, status);
    }
}

bool many_rows(const QCache &c, const QRows &r) { return (long long)r.rows * c.h_kv >= kManyRows; }

template <int GROUPS>
cudaError_t launch_write(const QCache &c, const QRows &r, bool fp8, int *status, cudaStream_t st) {
    const long long units = many_rows(c, r) ? ((long long)r.rows + kChunk - 1) / kChunk * c.h_kv * 2 : (long long)r.rows * c.h_kv;
    const unsigned grid = (unsigned)((units + kWarps - 1) / kWarps);
    const auto kernel = !many_rows(c, r) ? write_kernel<GROUPS>
                        : fp8            ? rows_kernel<GROUPS, true, false>
                                         : rows_kernel<GROUPS, false, false>;
    return launch_chained(kernel, grid, kWarps * 32, 0, st, c, r, status);
}

template <int GROUPS>
cudaError_t launch_read(const QCache &c, const QRows &r, bool fp8, int *status, cudaStream_t st) {
    const long long units = many_rows(c, r) ? ((long long)r.rows + kChunk - 1) / kChunk * c.h_kv * 2 : (long long)r.rows * c.h_kv;
    const unsigned grid = (unsigned)((units + kWarps - 1) / kWarps);
    const auto kernel = !many_rows(c, r) ? read_kernel<GROUPS>
                        : fp8            ? rows_kernel<GROUPS, true, true>
                                         : rows_kernel<GROUPS, false, true>;
    return launch_chained(kernel, grid, kWarps * 32, 0, st, c, r, status);
}

}  // namespace

cudaError_t launch_qcache_write(const QCache &c, const QRows &r, bool fp8, int *status, cudaStream_t st) {
    switch (c.groups) {
        case 4: return launch_write<4>(c, r, fp8, status, st);
        case 2: return launch_write<2>(c, r, fp8, status, st);
        default: return launch_write<1>(c, r, fp8, status, st);
    }
}

cudaError_t launch_qcache_read(const QCache &c, const QRows &r, bool fp8, int *status, cudaStream_t st) {
    switch (c.groups) {
        case 4: return launch_read<4>(c, r, fp8, status, st);
        case 2: return launch_read<2>(c, r, fp8, status, st);
        default: return launch_read<1>(c, r, fp8, status, st);
    }
}

}  // namespace fp
