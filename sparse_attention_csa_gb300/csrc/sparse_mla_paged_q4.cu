// Sparse MLA attention of new tokens over paged caches whose compressed rows
// are held in 4 bits (sm_103a). The window rows stay in bf16.
//
//     l_i = scale q.kv_i ; Z = sum e^(l_i - m) + e^(sink - m)
//     out = sum e^(l_i - m) kv_i / Z ; lse = m + ln Z
//
// One block a token and head; its warps share the keys, a lane holds 16 dims.
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "q4.cuh"

namespace csa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__global__ void __launch_bounds__(kThreads) sparse_mla_paged_q4_kernel(const __grid_constant__ MlaPagedArgs a) {
    __shared__ float acc_s[kWarps][512];
    __shared__ float m_s[kWarps], l_s[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t t = blockIdx.x, h = blockIdx.y;
    grid_dependency_wait();
    launch_dependents();
    const int32_t pos = __ldg(a.q_pos + t);
    const int32_t b = paged_seq(a.q_seq, a.batch, t, pos);
    if (b == -2) report_error(a.err, kErrCheck, kKerMlaPaged, 1);
    const __nv_bfloat16 *q = a.q + ((int64_t)t * a.H + h) * 512;
    float qf[16], acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        qf[i] = __bfloat162float(q[16 * lane + i]) * a.softmax_scale;
        acc[i] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    int32_t n_win = 0, start = 0, n_cmp = 0, vis = 0;
    if (b >= 0) {
        start = max(pos - a.window + 1, 0);
        n_win = pos - start + 1;
        if (a.cmp.base) {
            const int32_t cap = a.cmp.max_pages * a.cmp.page_size;
            vis = (int32_t)(((uint32_t)pos + 1u) / (uint32_t)a.cmp_ratio);
            if (vis > cap) {
                report_error(a.err, kErrCheck, kKerMlaPaged, 2);
                vis = cap;
            }
            n_cmp = a.idx ? (vis > 0 ? a.topk : 0) : vis;
        }
    }
    for (int64_t i = warp; i < (int64_t)n_win + n_cmp; i += kWarps) {
        const bool win = i < n_win;
        int32_t r = win ? start + (int32_t)i : (int32_t)(i - n_win);
        if (!win && a.idx) r = __ldg(a.idx + (int64_t)t * a.topk + r);
        if (r < 0 || (!win && r >= vis)) continue;
        const PagedRows &p = win ? a.ori : a.cmp;
        const uint32_t pg = (uint32_t)r / (uint32_t)p.page_size;
        const int32_t phys = pg < (uint32_t)p.max_pages ? __ldg(p.pages + (int64_t)b * p.max_pages + pg) : -1;
        if ((uint32_t)phys >= (uint32_t)p.num_pages) {
            if (phys != CSA_PAGE_EVICTED) report_error(a.err, kErrCheck, kKerMlaPaged, 3);
            continue;
        }
        const int64_t row = (int64_t)phys * p.page_size + (r - (int32_t)pg * p.page_size);
        uint4 v[2];
        if (win) {
            const uint4 *src = reinterpret_cast<const uint4 *>(p.base + row * 512) + 2 * lane;
            v[0] = __ldg(src);
            v[1] = __ldg(src + 1);
        } else {
            q4::sixteen(reinterpret_cast<const uint8_t *>(p.base) + row * q4::kRow, lane, v);
        }
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
        float k[16], s = 0.0f;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            k[2 * x] = __uint_as_float(w[x] << 16);
            k[2 * x + 1] = __uint_as_float(w[x] & 0xffff0000u);
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) s = fmaf(qf[x], k[x], s);
        s = warp_sum(s);
        const float mn = fmaxf(m, s), al = m == -INFINITY ? 0.0f : expf(m - mn), e = expf(s - mn);
        l = l * al + e;
#pragma unroll
        for (int x = 0; x < 16; ++x) acc[x] = fmaf(e, k[x], acc[x] * al);
        m = mn;
    }
#pragma unroll
    for (int x = 0; x < 16; ++x) acc_s[warp][16 * lane + x] = acc[x];
    if (lane == 0) {
        m_s[warp] = m;
        l_s[warp] = l;
    }
    __syncthreads();
    const float sk = a.sinks && b >= 0 ? __ldg(a.sinks + h) : -INFINITY;
    float M = sk, f[kWarps];
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, m_s[w]);
    float Z = sk == -INFINITY ? 0.0f : expf(sk - M);
    for (int w = 0; w < kWarps; ++w) {
        f[w] = m_s[w] == -INFINITY && l_s[w] == 0.0f ? 0.0f : expf(m_s[w] - M);
        Z = fmaf(l_s[w], f[w], Z);
    }
    for (int d = threadIdx.x; d < 512; d += kThreads) {
        float o = 0.0f;
        for (int w = 0; w < kWarps; ++w) o = fmaf(acc_s[w][d], f[w], o);
        a.out[((int64_t)t * a.H + h) * 512 + d] = __float2bfloat16_rn(Z == 0.0f ? 0.0f : o / Z);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(int64_t)t * a.H + h] = M + logf(Z);
}

}  // namespace

cudaError_t launch_sparse_mla_paged_q4(MlaPagedArgs a, cudaStream_t stream) {
    return launch_early(sparse_mla_paged_q4_kernel, dim3(a.T, a.H), dim3(kThreads), 0, stream, a);
}

}  // namespace csa
