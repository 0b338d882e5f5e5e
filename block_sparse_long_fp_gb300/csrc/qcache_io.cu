// fp_qcache_write and fp_qcache_read: rows of bf16 or e4m3 to the 4-bit cache
// and back.
//
// One warp per (row, kv head), four dims per lane, so a group of G dims is
// G / 4 neighbouring lanes and its extremes take log2(G / 4) shuffles.  Both
// are bound by memory: per (token, head) 512 bytes of bf16 on one side and
// 128 + 1024 / G bytes of cache on the other.
#include "qcache.cuh"

namespace fp {
namespace {

constexpr int kWarps = 8;

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

}  // namespace

cudaError_t launch_qcache_write(const QCache &c, const QRows &r, bool, int *status, cudaStream_t st) {
    const unsigned grid = (unsigned)(((long long)r.rows * c.h_kv + kWarps - 1) / kWarps);
    switch (c.groups) {
        case 4: return launch_chained(write_kernel<4>, grid, kWarps * 32, 0, st, c, r, status);
        case 2: return launch_chained(write_kernel<2>, grid, kWarps * 32, 0, st, c, r, status);
        default: return launch_chained(write_kernel<1>, grid, kWarps * 32, 0, st, c, r, status);
    }
}

cudaError_t launch_qcache_read(const QCache &c, const QRows &r, bool, int *status, cudaStream_t st) {
    const unsigned grid = (unsigned)(((long long)r.rows * c.h_kv + kWarps - 1) / kWarps);
    switch (c.groups) {
        case 4: return launch_chained(read_kernel<4>, grid, kWarps * 32, 0, st, c, r, status);
        case 2: return launch_chained(read_kernel<2>, grid, kWarps * 32, 0, st, c, r, status);
        default: return launch_chained(read_kernel<1>, grid, kWarps * 32, 0, st, c, r, status);
    }
}

}  // namespace fp
