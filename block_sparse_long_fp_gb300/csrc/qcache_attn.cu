// fp_qcache_attn: attention over the 4-bit cache.
//
// One warp per (query row, head) walks the keys with the running maximum and
// sum of a softmax in fp32, four dims per lane.
#include "qcache.cuh"

namespace fp {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

__global__ void __launch_bounds__(kWarps * 32) attn_kernel(QAttn a) {
    const long long unit = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
    if (unit >= (long long)a.total_q * a.h_q) return;
    if (unit == 0 && a.cu && a.cu[a.batch] > a.total_q) set_status(a.status, FP_ERR_DEVICE_BOUNDS);
    const int row = (int)(unit / a.h_q), head = (int)(unit % a.h_q), l = threadIdx.x & 31;
    int r, i, lq;
    if (a.cu) {
        int lo = 0, hi = a.batch - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu[mid] <= row) lo = mid; else hi = mid - 1;
        }
        r = lo;
        i = row - a.cu[r];
        lq = a.cu[r + 1] - a.cu[r];
    } else {
        r = row / a.max_q;
        i = row % a.max_q;
        lq = a.max_q;
    }
    if (r >= a.batch || i < 0 || i >= lq) return;
    int len = a.seqlens_k[r];
    if (len < 0 || len > (long long)a.max_pages * a.c.page_size) {
        set_status(a.status, FP_ERR_DEVICE_BOUNDS);
        len = 0;
    }
    const int keys = min(len, len - lq + i + 1);
    const long long at = row * a.q_stride_tok + head * a.q_stride_head + 4 * l;
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (a.q_scale) {
            __nv_fp8_e4m3 x;
            x.__x = static_cast<const unsigned char *>(a.q)[at + e];
            q[e] = (float)x * a.q_scale[head];
        } else {
            q[e] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[at + e]);
        }
    }
    const int groups = a.c.groups, lane_group = l * groups / 32, kv = head / a.g;
    for (int t = 0; t < keys; ++t) {
        const int page = a.block_table[(long long)r * a.max_pages + t / a.c.page_size];
        float s = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
        if (page >= 0 && page < a.c.num_pages) {
            const unsigned char *chunk = qcache_chunk(a.c, page * a.c.page_size + t % a.c.page_size, kv);
            const int tt = t % kChunk;
            const uint32_t kw = *reinterpret_cast<const uint16_t *>(chunk + k_code_off(tt, l));
            const uint32_t vw = *reinterpret_cast<const uint16_t *>(chunk + v_code_off(tt, l));
            const __half *ks = reinterpret_cast<const __half *>(chunk + k_step_off(tt, lane_group, groups));
            const __half *vs = reinterpret_cast<const __half *>(chunk + v_step_off(tt, lane_group, groups));
            const float s_k = __half2float(ks[0]), m_k = __half2float(ks[16 * groups]);
            const float s_v = __half2float(vs[0]), m_v = __half2float(vs[16 * groups]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s = fmaf(q[e], fmaf(s_k, (float)((kw >> (4 * e)) & 15u), m_k), s);
                v[e] = fmaf(s_v, (float)((vw >> (4 * e)) & 15u), m_v);
            }
        } else if (l == 0) {
            set_status(a.status, FP_ERR_DEVICE_BOUNDS);
        }
#pragma unroll
        for (int d = 16; d; d /= 2) s += __shfl_xor_sync(~0u, s, d);
        s *= a.scale * kLog2e;
        const float top = fmaxf(m, s), keep = exp2f(m - top), p = exp2f(s - top);
        m = top;
        sum = fmaf(sum, keep, p);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = fmaf(o[e], keep, p * v[e]);
    }
    const float inv = keys > 0 ? 1.f / sum : 0.f;
    __nv_bfloat16 *out = a.out + ((long long)row * a.h_q + head) * kHeadDim + 4 * l;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = __float2bfloat16_rn(o[e] * inv);
    if (a.lse && l == 0) a.lse[(long long)head * a.total_q + row] = keys > 0 ? (m + log2f(sum)) / kLog2e : -INFINITY;
}

}  // namespace

size_t qcache_attn_scratch_bytes(const QAttn &) { return 16; }

cudaError_t launch_qcache_attn(const QAttn &a, void *, cudaStream_t st) {
    const long long units = (long long)a.total_q * a.h_q;
    attn_kernel<<<(unsigned)((units + kWarps - 1) / kWarps), kWarps * 32, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace fp
