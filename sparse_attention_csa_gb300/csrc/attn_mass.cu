// The attention weight that cached compressed rows received (sm_103a):
//
//     out[b, j] = mass[b, j] + sum over the tokens t of sequence b that attend
//                 row j, and their heads h, of e^(scale q[t,h].k_j - lse[t,h])
//
// Two kernels. The first leaves the weight of every (token, key slot), heads
// summed, in the workspace; the second adds a sequence's tokens up in an order
// that does not depend on the launch. Listed rows are added in shared memory as
// fixed-point numbers, whose sums have no order (a row may be listed twice).
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "q4.cuh"

namespace csa {

namespace {

// Visible compressed rows of token t, and its sequence (-1: none).
__device__ __forceinline__ int32_t visible_rows(const MassArgs &a, int32_t t, int32_t *seq, bool report) {
    const int32_t pos = __ldg(a.q_pos + t);
    const int32_t b = paged_seq(a.q_seq, a.batch, t, pos);
    *seq = b < 0 ? -1 : b;
    if (b < 0) {
        if (b == -2 && report) report_error(a.err, kErrCheck, kKerMass, 1);
        return 0;
    }
    const int32_t n = (int32_t)(((uint32_t)pos + 1u) / (uint32_t)a.cmp_ratio);
    if (n > a.max_rows) {
        if (report) report_error(a.err, kErrCheck, kKerMass, 2);
        return a.max_rows;
    }
    return n;
}

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) attn_weight_kernel(const __grid_constant__ MassArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t t = blockIdx.x;
    grid_dependency_wait();
    launch_dependents();
    int32_t b;
    const int32_t vis = visible_rows(a, t, &b, true);
    const int32_t slots = a.idx ? (vis > 0 ? a.topk : 0) : vis;
    float *out = a.weights + t * a.slot_pad;
    for (int64_t i = (int64_t)blockIdx.y * 8 + warp; i < slots; i += 8 * gridDim.y) {
        const int32_t r = a.idx ? __ldg(a.idx + (int64_t)t * a.topk + i) : (int32_t)i;
        float sum = 0.0f;
        if (r >= 0 && r < vis) {
            const uint32_t pg = (uint32_t)r / (uint32_t)a.cmp.page_size;
            const int32_t phys = __ldg(a.cmp.pages + (int64_t)b * a.cmp.max_pages + pg);
            if ((uint32_t)phys < (uint32_t)a.cmp.num_pages) {
                const int64_t row = (int64_t)phys * a.cmp.page_size + (r - (int32_t)pg * a.cmp.page_size);
                uint4 v[2];
                if (a.q4) {
                    q4::sixteen(reinterpret_cast<const uint8_t *>(a.cmp.base) + row * q4::kRow, lane, v);
                } else {
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.cmp.base + row * 512) + 2 * lane;
                    v[0] = __ldg(src);
                    v[1] = __ldg(src + 1);
                }
                const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
                for (int h = 0; h < a.H; ++h) {
                    const __nv_bfloat16 *q = a.q + ((int64_t)t * a.H + h) * 512 + 16 * lane;
                    float s = 0.0f;
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        s = fmaf(__bfloat162float(q[2 * x]), __uint_as_float(w[x] << 16), s);
                        s = fmaf(__bfloat162float(q[2 * x + 1]), __uint_as_float(w[x] & 0xffff0000u), s);
                    }
                    s = warp_sum(s);
                    const float lse = __ldg(a.lse + (int64_t)t * a.H + h);
                    if (lse != -INFINITY) sum += expf(s * a.softmax_scale - lse);
                }
            } else if (phys != CSA_PAGE_EVICTED) {
                report_error(a.err, kErrCheck, kKerMass, 3);
            }
        }
        // NaN counts as 0; more than one a head only an lse that is not the attention's can give
        if (lane == 0) out[i] = sum <= (float)a.H ? sum : sum > (float)a.H ? (float)a.H : 0.0f;
    }
}

// out = mass + the weights: a block takes kRows rows of one sequence.
constexpr int kRows = 4096;

__global__ void __launch_bounds__(kThreads) attn_mass_kernel(const __grid_constant__ MassArgs a) {
    __shared__ unsigned long long acc[kRows];
    const int32_t b = blockIdx.y, r0 = blockIdx.x * kRows, n = min(kRows, a.max_rows - r0);
    grid_dependency_wait();
    launch_dependents();
    for (int i = threadIdx.x; i < n; i += kThreads) acc[i] = 0;
    __syncthreads();
    for (int32_t t = 0; t < a.T; ++t) {
        int32_t seq;
        const int32_t vis = visible_rows(a, t, &seq, false);
        if (seq != b) continue;
        const int32_t slots = a.idx ? (vis > 0 ? a.topk : 0) : vis;
        for (int32_t i = threadIdx.x; i < slots; i += kThreads) {
            const int32_t r = a.idx ? __ldg(a.idx + (int64_t)t * a.topk + i) : i;
            if (r >= vis || r < r0 || r >= r0 + n) continue;
            atomicAdd(&acc[r - r0], __float2ull_rn(a.weights[t * a.slot_pad + i] * a.fixed));
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int64_t o = (int64_t)b * a.max_rows + r0 + i;
        const float old = a.mass ? a.mass[o] : 0.0f;
        a.out[o] = acc[i] ? old + (float)((double)acc[i] / (double)a.fixed) : old;
    }
}

}  // namespace

int64_t mass_slot_pad(int64_t slots) { return (slots + 127) & ~(int64_t)127; }

size_t mass_workspace_bytes(int32_t T, int64_t slots) {
    return T > 0 ? (size_t)T * (size_t)mass_slot_pad(slots) * 4 : 0;
}

cudaError_t launch_attn_mass(MassArgs a, cudaStream_t stream) {
    if (a.T > 0) {
        const cudaError_t e = launch_early(attn_weight_kernel, dim3(a.T, 64), dim3(kThreads), 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    if (a.batch == 0 || a.max_rows == 0) return cudaSuccess;
    return launch_early(attn_mass_kernel, dim3((a.max_rows + kRows - 1) / kRows, a.batch), dim3(kThreads), 0,
                        stream, a);
}

}  // namespace csa
