// Rows to and from a paged cache that holds them in 4 bits (sm_103a).
//
// Append, for a row x (its last dims rotated first):
//     top_g = max |x_d| over the 16 dims of group g (finite ones),
//     2^e: e = floor(log2(max_g top_g / 6)) - 7 within [-100, 100],
//     s_g = top_g / 6 / 2^e to e4m3, largest finite 448,
//     code_d = |x_d| / (s_g 2^e) to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6,
// ties to the even code. The quotient rounded to 32 bits decides as the exact one
// does: midpoints are such numbers, and no other quotient by a scale of four
// significant bits rounds to one of them (|x_d| one unit away is off by 2^-23 /
// its mantissa, relative, half a unit of the quotient by 2^-24 / the
// quotient's). It is the product with the scale's reciprocal and Markstein's
// correction by the exact remainder. The rotary dims are rounded to bf16. A
// group with a value that is not finite gets a NaN scale and reads as NaN.
//
// A warp takes a row, a lane one group: the lanes' 32 x 16 dims are the row's 28
// groups and 64 rotary dims, so the only exchange is one maximum. (Two or four
// rows a warp took registers, hence warps on an SM: 16368 rows and their reading
// back, in blocks of 256 threads, 15.8 us with one, 16.4 and 22.7. Blocks of 128
// threads 15.2; warps that take rows in turn, the next one's on its way, spill.)
//
// The append is bound by the latency of a row's way, two dependent look-ups ahead
// of its first store, beside 420 instructions that issue 42 % of the time (16368
// bf16 rows, 23 MB: 9 us of the 15.3); the read by memory and the look-up (40955
// rows, 58 MB: 12.6 us, 4.6 TB/s).
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "q4.cuh"
#include "rope_angle.cuh"

namespace csa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = q4::kDims / q4::kGroup;

// Row of the pool, or -1: padding, or absent (recorded unless evicted on purpose).
__device__ __forceinline__ int64_t find_row(const Q4RowsArgs &a, int64_t t, bool writes) {
    if (t >= a.T) return -1;
    const int32_t p = __ldg(a.row_pos + t);
    const int32_t b = paged_seq(a.row_seq, a.batch, (int32_t)t, p);
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

// Two values as codes: `a` in the low four bits.
__device__ __forceinline__ uint32_t two_codes(float a, float b) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b));
    return r;
}

// x / s rounded to 32 bits, inv being 1 / s rounded so (0 with s 0: 0). A zero
// keeps its sign.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
    const float q = x * inv;
    return fmaf(-fmaf(q, s, -x), inv, q);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 12) cache_append_q4_kernel(const __grid_constant__ Q4RowsArgs a) {
    __shared__ alignas(16) float tail_s[kWarps][64];
    __shared__ uint64_t turns_s[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *tail = tail_s[warp];
    grid_dependency_wait();
    launch_dependents();
    const int np = a.n / 2;
    if (warp == 0 && lane < np) turns_s[lane] = fixed_turns(__ldg(a.inv_freq + lane));  // once: 64-bit products
    const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    float x[16];
    if (t < a.T) load16<T, VEC>(static_cast<const T *>(a.rows) + t * a.row_stride + 16 * lane, x);
    const int64_t slot = find_row(a, t, true);
    __syncthreads();
    if (slot < 0) return;
    const uint64_t turns = lane < np ? turns_s[lane] : 0;
    // the pair of rotary dims that this lane turns, within the last 64
    const int d0 = a.off - q4::kDims + (a.half ? lane : 2 * lane), d1 = d0 + (a.half ? np : 1);
    uint8_t *row = a.cache + slot * q4::kRow;
    // the largest magnitude, by its bits; of the finite values
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    const bool fine = top < 0x7f800000u;
    if (!fine && lane < kGroups) {
        top = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t m = __float_as_uint(x[i]) & 0x7fffffffu;
            top = max(top, m < 0x7f800000u ? m : 0u);
            x[i] = copysignf(0.0f, x[i]);
        }
    }
    const uint32_t all = __reduce_max_sync(0xffffffffu, lane < kGroups ? top : 0u);
    // floor(log2(all / 6)) - 7: a sixth of a mantissa below 1.5 is below 1 / 4
    const int e = min(max((int)(all >> 23) - 127 - 3 + ((all & 0x7fffffu) >= 0x400000u) - 7, q4::kMinExp),
                      q4::kMaxExp);
    if (lane < kGroups) {
        const float scaled = fine ? quotient(__uint_as_float(top) * q4::pow2(-e), 6.0f, 1.0f / 6.0f) : 0.0f;
        uint8_t s8 = (uint8_t)__nv_cvt_float_to_fp8(scaled, __NV_SATFINITE, __NV_E4M3);
        const float s = q4::scales2(s8).x * q4::pow2(e);
        const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;  // a group that vanished, or without a scale: zeros
        if (!fine) s8 = 0x7f;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = quotient(x[i], s, inv);
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float *v = x + 8 * h;
            w[h] = two_codes(v[0], v[2]) | two_codes(v[4], v[6]) << 8 | two_codes(v[1], v[3]) << 16 |
                   two_codes(v[5], v[7]) << 24;
        }
        reinterpret_cast<uint2 *>(row)[lane] = make_uint2(w[0], w[1]);
        row[q4::kScales + lane] = s8;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4 *>(tail)[4 * (lane - kGroups) + i] =
                make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
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
}

// A lane has two pieces of eight dims, 256 dims apart: a warp writes 512 bytes
// at a time.
template <int ROWS>
__global__ void __launch_bounds__(kThreads) cache_read_q4_kernel(const __grid_constant__ Q4RowsArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    launch_dependents();
    const int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * ROWS;
    const int64_t found = lane < ROWS ? find_row(a, t0 + lane, false) : -1;
    q4::Eight v[ROWS][2];
#pragma unroll
    for (int y = 0; y < ROWS; ++y) {
        const int64_t slot = __shfl_sync(0xffffffffu, found, y);
#pragma unroll
        for (int h = 0; h < 2; ++h) v[y][h].load(slot < 0 ? nullptr : a.cache + slot * q4::kRow, lane + 32 * h);
    }
#pragma unroll
    for (int y = 0; y < ROWS; ++y) {
        if (t0 + y >= a.T) break;
        uint4 *out = reinterpret_cast<uint4 *>(a.out + (t0 + y) * 512) + lane;
        out[0] = v[y][0].values(lane);
        out[32] = v[y][1].values(lane + 32);
    }
}

unsigned row_blocks(int32_t T, int rows) { return (unsigned)(((int64_t)T + kWarps * rows - 1) / (kWarps * rows)); }

template <typename T, bool VEC>
cudaError_t append_q4(const Q4RowsArgs &a, cudaStream_t stream) {
    return launch_early(cache_append_q4_kernel<T, VEC>, dim3(row_blocks(a.T, 1)), dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_cache_append_q4(const Q4RowsArgs &a, cudaStream_t stream) {
    const int es = a.f32 ? 4 : 2;
    const bool vec = ((reinterpret_cast<uintptr_t>(a.rows) | (uintptr_t)(a.row_stride * es)) & 15u) == 0;
    if (a.f32) return vec ? append_q4<float, true>(a, stream) : append_q4<float, false>(a, stream);
    return vec ? append_q4<__nv_bfloat16, true>(a, stream) : append_q4<__nv_bfloat16, false>(a, stream);
}

cudaError_t launch_cache_read_q4(const Q4RowsArgs &a, cudaStream_t stream) {
    int sms;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    // two rows a warp while that leaves an SM 32 warps: 16384, 40955 and 120000 rows
    // 6.4, 12.5 and 30.1 us, with one 6.6, 13.1 and 33.6; 64 and 6000 rows 1.9 and
    // 4.1 us, with one 1.6 and 3.7
    return a.T >= 64 * sms
               ? launch_early(cache_read_q4_kernel<2>, dim3(row_blocks(a.T, 2)), dim3(kThreads), 0, stream, a)
               : launch_early(cache_read_q4_kernel<1>, dim3(row_blocks(a.T, 1)), dim3(kThreads), 0, stream, a);
}

}  // namespace csa
