// Rows to and from a paged cache that holds them in 4 bits (sm_103a).
//
// Append, for a row x (its last dims rotated first):
//     top_g = max |x_d| over the 16 dims of group g (finite ones),
//     2^e: e = floor(log2(max_g top_g / 6)) - 7 within [-100, 100],
//     s_g = top_g / 6 / 2^e to e4m3, largest finite 448,
//     code_d = |x_d| / (s_g 2^e) to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6,
// ties to the even code. The nearest is found by comparing |x_d| with the seven
// midpoints times the scale, which are exact products: a quotient would round
// once more and could cross a midpoint. The rotary dims are rounded to bf16. A
// group with a value that is not finite gets a NaN scale and reads as NaN.
//
// A warp takes a row, a lane one group: the lanes' 32 x 16 dims are the row's
// 28 groups and 64 rotary dims, so the only exchange is one maximum.
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "q4.cuh"
#include "rope_angle.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = q4::kDims / q4::kGroup;

// Row of the pool, or -1: padding, or absent (recorded unless evicted on purpose).
__device__ __forceinline__ int64_t find_row(const Q4RowsArgs &a, int32_t t, bool writes) {
    const int32_t p = __ldg(a.row_pos + t);
    const int32_t b = paged_seq(a.row_seq, a.batch, t, p);
    if (b == -2) report_error(a.err, kErrCheck, kKerCacheQ4, 1);
    if (b < 0) return -1;
    const uint32_t pg = (uint32_t)p / (uint32_t)a.page_size;
    const int32_t phys = pg < (uint32_t)a.max_pages ? __ldg(a.pages + (int64_t)b * a.max_pages + pg) : -1;
    if ((uint32_t)phys >= (uint32_t)a.num_pages) {
        if (writes || phys != CSA_PAGE_EVICTED) report_error(a.err, kErrCheck, kKerCacheQ4, 2);
        return -1;
    }
    return (int64_t)phys * a.page_size + (p - (int32_t)pg * a.page_size);
}

// 16 dims from p; VEC: p is 16-byte aligned
template <typename T, bool VEC>
__device__ __forceinline__ void load16(const T *p, float (&x)[16]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = (float)p[i];
    } else if constexpr (sizeof(T) == 2) {
        const uint4 v[2] = {__ldg(reinterpret_cast<const uint4 *>(p)), __ldg(reinterpret_cast<const uint4 *>(p) + 1)};
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(p) + i);
            x[4 * i] = v.x;
            x[4 * i + 1] = v.y;
            x[4 * i + 2] = v.z;
            x[4 * i + 3] = v.w;
        }
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) cache_append_q4_kernel(const __grid_constant__ Q4RowsArgs a) {
    __shared__ float tail_s[kWarps][64];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *tail = tail_s[warp];
    grid_dependency_wait();
    launch_dependents();
    const int np = a.n / 2;
    const uint64_t turns = lane < np ? fixed_turns(__ldg(a.inv_freq + lane)) : 0;
    // the pair of rotary dims that this lane turns, within the last 64
    const int d0 = a.off - q4::kDims + (a.half ? lane : 2 * lane), d1 = d0 + (a.half ? np : 1);
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T; t += (int64_t)gridDim.x * kWarps) {
        float x[16];
        load16<T, VEC>(static_cast<const T *>(a.rows) + t * a.row_stride + 16 * lane, x);
        const int64_t slot = find_row(a, (int32_t)t, true);
        if (slot < 0) continue;
        uint8_t *row = a.cache + slot * q4::kRow;
        float top = 0.0f;
        bool fine = true;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float m = fabsf(x[i]);
            const bool f = m <= 3.402823466e38f;
            fine &= f;
            top = fmaxf(top, f ? m : 0.0f);
        }
        const float all = warp_max(lane < kGroups ? top : 0.0f);
        const int e = min(max((int)((__float_as_uint(__fdiv_rn(all, 6.0f)) >> 23) & 255u) - 127 - 7,
                              q4::kMinExp), q4::kMaxExp);
        if (lane < kGroups) {
            const uint8_t s8 = fine ? (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(top, 6.0f) * q4::pow2(-e),
                                                                     __NV_SATFINITE, __NV_E4M3)
                                    : (uint8_t)0x7f;
            const float s = q4::scales2(s8).x * q4::pow2(e);
            uint32_t w[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float m = fabsf(x[i]);
                uint32_t code = (m > 0.25f * s) + (m >= 0.75f * s) + (m > 1.25f * s) + (m >= 1.75f * s) +
                                (m > 2.5f * s) + (m >= 3.5f * s) + (m > 5.0f * s);
                if (!(s > 0.0f)) code = 0;  // a group that vanished, or without a scale
                code |= (__float_as_uint(x[i]) >> 31) << 3;
                w[i >> 3] |= code << (4 * ((i >> 1) & 3) + 16 * (i & 1));
            }
            reinterpret_cast<uint2 *>(row)[lane] = make_uint2(w[0], w[1]);
            row[q4::kScales + lane] = s8;
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) tail[16 * (lane - kGroups) + i] = x[i];
            if (lane == kGroups) *reinterpret_cast<uint32_t *>(row + q4::kExp) = (uint32_t)(e + 127);
        }
        __syncwarp();
        if (lane < np) {
            const float2 cs = cos_sin((int64_t)__ldg(a.row_pos + t) * a.pos_stride, turns, 1.0f, a.mscale);
            const float u = tail[d0], v = tail[d1];
            tail[d0] = fmaf(u, cs.x, -v * cs.y);
            tail[d1] = fmaf(v, cs.x, u * cs.y);
        }
        __syncwarp();
        reinterpret_cast<__nv_bfloat162 *>(row + q4::kTail)[lane] =
            __floats2bfloat162_rn(tail[2 * lane], tail[2 * lane + 1]);
        __syncwarp();
    }
}

__global__ void __launch_bounds__(kThreads) cache_read_q4_kernel(const __grid_constant__ Q4RowsArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    launch_dependents();
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T; t += (int64_t)gridDim.x * kWarps) {
        const int64_t slot = find_row(a, (int32_t)t, false);
        uint4 v[2] = {};
        if (slot >= 0) q4::sixteen(a.cache + slot * q4::kRow, lane, v);
        uint4 *out = reinterpret_cast<uint4 *>(a.out + t * 512) + 2 * lane;
        out[0] = v[0];
        out[1] = v[1];
    }
}

unsigned row_blocks(int32_t T) { return (unsigned)(((int64_t)T + kWarps - 1) / kWarps); }

}  // namespace

cudaError_t launch_cache_append_q4(const Q4RowsArgs &a, cudaStream_t stream) {
    const int es = a.f32 ? 4 : 2;
    const bool vec = ((reinterpret_cast<uintptr_t>(a.rows) | (uintptr_t)(a.row_stride * es)) & 15u) == 0;
    const dim3 grid(row_blocks(a.T)), block(kThreads);
    if (a.f32)
        return vec ? launch_early(cache_append_q4_kernel<float, true>, grid, block, 0, stream, a)
                   : launch_early(cache_append_q4_kernel<float, false>, grid, block, 0, stream, a);
    return vec ? launch_early(cache_append_q4_kernel<__nv_bfloat16, true>, grid, block, 0, stream, a)
               : launch_early(cache_append_q4_kernel<__nv_bfloat16, false>, grid, block, 0, stream, a);
}

cudaError_t launch_cache_read_q4(const Q4RowsArgs &a, cudaStream_t stream) {
    return launch_early(cache_read_q4_kernel, dim3(row_blocks(a.T)), dim3(kThreads), 0, stream, a);
}

}  // namespace csa
