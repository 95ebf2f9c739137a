// Rotary positions over part of a head, and the same rotation on the way into
// a paged row cache (sm_103a).
//
//     theta = p f_i (radians; p the position, f_i in 64 bits)
//     y_a = m (x_a cos theta - x_b sin theta)
//     y_b = m (x_b cos theta + x_a sin theta)
// for the pairs (a, b) of the rotary part: neighbours (interleaved) or i and
// i + n/2 (half). The inverse turns by -theta, which for m > 0 is the
// transpose of the forward map, hence also its backward.
//
// Memory bound: a block first turns its tokens' angles into a shared table of
// (cos, sin), computed once for all heads of a token, and then streams 16-byte
// pieces. (Several pieces a thread in flight at once cost more in registers,
// hence blocks on an SM, than they gained: 8192 x 64 heads of 512 bf16 dims,
// 1.07 GB, 247 us with four, 166 us with one.)
//
// Angles need 64 bits (at p = 2^20 a 32-bit product p f is off by up to 2^-5
// radians), but 64-bit floating point is slow here. So a block turns each
// frequency once into a fraction of a turn per position in fixed point, in
// units of 2^-64 turns; p times that, modulo 2^64, is the angle without its
// whole turns: three integer multiplications that add no error to the
// frequency's (f / 2 pi is a product in 64 bits with a rounded constant: 2^-52
// of it, times p, so 2^-34 turns at p = 2^20 and f = 1). Its upper 32 bits, as
// a signed fraction, are half a turn at most: 24 of them go through sincospif
// as a float, exactly, and the other 8 turn its result by their own angle,
// below 2^-22 radians (a float of all 32 would be off by 2^-23.3 radians, as
// much as sincospif itself: factors up to 2^20 positions were off by up to
// 1.16e-7, and are by 8.0e-8; no case got slower).
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "rope_angle.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kTable = 2048;    // (cos, sin) pairs per block: 16 KB
constexpr int kMaxRows = 128;   // tokens per block
constexpr int kMaxPairs = 512;  // rope_dim <= 1024
constexpr int kPieces = 4;      // copied pieces a thread of the append takes

// V consecutive elements <-> fp32
template <typename T, int V>
__device__ __forceinline__ void load_v(const T *p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = (float)p[0];
    } else if constexpr (sizeof(T) == 2) {
        static_assert(V == 8, "16 bytes of bf16");
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 u = reinterpret_cast<const float4 *>(p)[i];
            v[4 * i] = u.x;
            v[4 * i + 1] = u.y;
            v[4 * i + 2] = u.z;
            v[4 * i + 3] = u.w;
        }
    }
}

// rounded to nearest even once, on the way out
template <typename T, int V>
__device__ __forceinline__ void store_v(T *p, const float (&v)[V]) {
    if constexpr (V == 1) {
        p[0] = (T)v[0];
    } else if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            reinterpret_cast<float4 *>(p)[i] =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
}

// V pairs, from pair j of the rotary part (x and y point at its first
// element), turned by tab[j ..]. Interleaved: elements 2j .. 2j + 2V; half:
// j .. j + V and n/2 + j .. n/2 + j + V.
template <typename Ti, typename To, int V, bool HALF>
__device__ __forceinline__ void turn_pairs(const Ti *x, To *y, const float2 *tab, int j, int n) {
    const int i0 = HALF ? j : 2 * j, i1 = HALF ? n / 2 + j : 2 * j + V;
    float u[V], v[V];
    load_v<Ti, V>(x + i0, u);
    load_v<Ti, V>(x + i1, v);
    auto one = [&](float &a, float &b, float2 cs) {
        const float ra = fmaf(a, cs.x, -b * cs.y), rb = fmaf(b, cs.x, a * cs.y);
        a = ra;
        b = rb;
    };
    if constexpr (HALF || V == 1) {
#pragma unroll
        for (int e = 0; e < V; ++e) one(u[e], v[e], tab[j + e]);
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            one(u[e], u[e + 1], tab[j + e / 2]);
            one(v[e], v[e + 1], tab[j + V / 2 + e / 2]);
        }
    }
    store_v<To, V>(y + i0, u);
    store_v<To, V>(y + i1, v);
}

__global__ void rope_freqs_kernel(RopeFreqsArgs a) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x, half = a.rope_dim / 2;
    if (i >= half) return;
    const double f = pow(a.theta, -2.0 * i / a.rope_dim);
    double g = f / a.factor;
    if (a.original_len > 0) {
        // By parts: pairs turning more than beta_fast times over the original
        // length keep their frequency, those turning less than beta_slow times
        // are stretched by the factor, and a ramp over the pair index joins them.
        const double two_pi = 6.283185307179586477, lt = 2.0 * log(a.theta);
        const double lo = floor(a.rope_dim * log(a.original_len / (a.beta_fast * two_pi)) / lt);
        const double hi = ceil(a.rope_dim * log(a.original_len / (a.beta_slow * two_pi)) / lt);
        const double l = fmax(lo, 0.0), h = fmin(hi, a.rope_dim - 1.0);
        const double ramp = fmin(fmax((i - l) / fmax(h - l, 1e-3), 0.0), 1.0);
        g = g * ramp + f * (1.0 - ramp);
    }
    a.inv_freq[i] = g;
}

// Block: `tb` tokens x `hb` heads.
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a, int tb, int hb) {
    __shared__ float2 tab[kTable];
    __shared__ uint64_t turns[kMaxPairs];
    const int32_t t0 = blockIdx.x * tb, h0 = blockIdx.y * hb;
    const int nt = min(tb, a.T - t0), nh = min(hb, a.H - h0), np = a.n / 2;
    const float sign = a.inverse ? -1.0f : 1.0f;
    grid_dependency_wait();
    launch_dependents();
    const T *x = static_cast<const T *>(a.x) + t0 * a.x_stride + (int64_t)h0 * a.D;
    T *y = static_cast<T *>(a.out) + t0 * a.out_stride + (int64_t)h0 * a.D;
    const int rows = nt * nh;
    for (int i = threadIdx.x; i < np; i += kThreads) turns[i] = fixed_turns(__ldg(a.inv_freq + i));
    if (a.x != a.out) {  // first: the copies need no angles
        const int uc = (a.D - a.n) / V;  // copied units per (token, head)
        for (int i = threadIdx.x; i < rows * uc; i += kThreads) {
            const int row = i / uc, u = i - row * uc, r = row / nh, h = row - r * nh;
            const int64_t o = (int64_t)h * a.D + (u * V < a.off ? u * V : u * V + a.n);
            float v[V];
            load_v<T, V>(x + r * a.x_stride + o, v);
            store_v<T, V>(y + r * a.out_stride + o, v);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * np; i += kThreads) {
        const int r = i / np;
        const int32_t t = t0 + r;
        int64_t p = 0;
        if (a.positions) {
            p = __ldg(a.positions + t);
        } else {
            const int32_t b = find_segment(a.cu, a.batch, t);
            if (b >= 0)
                p = t - __ldg(a.cu + b);
            else
                report_error(a.err, kErrCheck, kKerRope, 1);
        }
        tab[i] = cos_sin(p * a.pos_stride, turns[i - r * np], sign, a.mscale);
    }
    __syncthreads();
    const int ur = np / V;  // turned units
    for (int i = threadIdx.x; i < rows * ur; i += kThreads) {
        const int row = i / ur, u = i - row * ur, r = row / nh, h = row - r * nh;
        const int64_t o = (int64_t)h * a.D + a.off;
        turn_pairs<T, T, V, HALF>(x + r * a.x_stride + o, y + r * a.out_stride + o, tab + r * np, u * V,
                                  a.n);
    }
}

// Block: `tb` rows. Rows whose slot cannot be named are skipped.
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const __grid_constant__ AppendArgs a, int tb) {
    __shared__ float2 tab[kTable];
    __shared__ uint64_t turns[kMaxPairs];
    __shared__ int64_t slot[kMaxRows];
    const int32_t t0 = blockIdx.x * tb;
    const int nt = min(tb, a.T - t0), np = a.n / 2;
    grid_dependency_wait();
    launch_dependents();
    const T *x = static_cast<const T *>(a.rows) + t0 * a.row_stride;
    const int ur = np / V, uc = (a.D - a.n) / V;
    // fp32: the dims that are only copied are on their way while the slots are
    // found (8005 rows of 512: 8.4 us, 9.4 without). bf16 rows, half as long,
    // lose by it (16368 rows of 512: 16 us, 10.9 without).
    constexpr int kAhead = sizeof(T) == 4 ? kPieces : 0;
    float v[kAhead + 1][V];
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
        const int i = threadIdx.x + z * kThreads;
        if (i < nt * uc) {
            const int r = i / uc, u = i - r * uc;
            load_v<T, V>(x + r * a.row_stride + (u * V < a.off ? u * V : u * V + a.n), v[z]);
        }
    }
    for (int r = threadIdx.x; r < nt; r += kThreads) {
        const int32_t p = __ldg(a.row_pos + t0 + r);
        const int32_t b = paged_seq(a.row_seq, a.batch, t0 + r, p);
        int64_t s = -1;
        if (b >= 0) s = paged_row({a.cache, a.pages, a.num_pages, a.page_size, a.max_pages}, b, p);
        if (b == -2 || (b >= 0 && s < 0)) report_error(a.err, kErrCheck, kKerAppend, b < 0 ? 1 : 2);
        slot[r] = s;
    }
    for (int i = threadIdx.x; i < np; i += kThreads) turns[i] = fixed_turns(__ldg(a.inv_freq + i));
    __syncthreads();
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
        const int i = threadIdx.x + z * kThreads;
        if (i < nt * uc) {
            const int r = i / uc, u = i - r * uc;
            if (slot[r] >= 0)
                store_v<__nv_bfloat16, V>(a.cache + slot[r] * a.D + (u * V < a.off ? u * V : u * V + a.n),
                                          v[z]);
        }
    }
    for (int i = threadIdx.x + kAhead * kThreads; i < nt * uc; i += kThreads) {
        const int r = i / uc, u = i - r * uc;
        const int e = u * V < a.off ? u * V : u * V + a.n;
        if (slot[r] < 0) continue;
        float w[V];
        load_v<T, V>(x + r * a.row_stride + e, w);
        store_v<__nv_bfloat16, V>(a.cache + slot[r] * a.D + e, w);
    }
    if (np == 0) return;
    for (int i = threadIdx.x; i < nt * np; i += kThreads) {
        const int r = i / np;
        const int64_t p = __ldg(a.row_pos + t0 + r);
        tab[i] = cos_sin(p * a.pos_stride, turns[i - r * np], 1.0f, a.mscale);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * ur; i += kThreads) {
        const int r = i / ur, u = i - r * ur;
        if (slot[r] >= 0)
            turn_pairs<T, __nv_bfloat16, V, HALF>(x + r * a.row_stride + a.off,
                                                  a.cache + slot[r] * a.D + a.off, tab + r * np, u * V, a.n);
    }
}

bool aligned(const void *p, int64_t stride_bytes) {
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride_bytes) & 15u) == 0;
}

// Blocks of `each` for n things, n up to 2^31 - 1.
unsigned blocks(int32_t n, int each) { return (unsigned)(((int64_t)n + each - 1) / each); }

}  // namespace

cudaError_t launch_rope_freqs(const RopeFreqsArgs &a, cudaStream_t stream) {
    rope_freqs_kernel<<<(a.rope_dim / 2 + 63) / 64, 64, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream) {
    const int es = a.f32 ? 4 : 2, V = 16 / es;
    // 16-byte pieces when every row and both parts of it start on 16 bytes
    const bool vec = aligned(a.x, a.x_stride * es) && aligned(a.out, a.out_stride * es) &&
                     a.D % V == 0 && a.off % V == 0 && a.n % (2 * V) == 0;
    const int units = (a.x == a.out ? a.n : a.D) / (vec ? V : 1);
    int sms;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    // rows (token, head) per block: about sixteen units a thread, fewer while
    // that leaves an SM with less than two blocks
    int64_t rows = max(1, 16 * kThreads / max(units, 1));
    rows = min(rows, max((int64_t)1, (int64_t)a.T * a.H / (2 * sms)));
    const int hb = (int)min((int64_t)a.H, rows);
    const int tb = (int)max((int64_t)1, min(min(rows / hb, (int64_t)kMaxRows), (int64_t)(kTable / (a.n / 2))));
    const dim3 grid(blocks(a.T, tb), blocks(a.H, hb));
#define CSA_ROPE(T, VV)                                                          \
    do {                                                                         \
        if (a.half)                                                              \
            return launch_early(rope_kernel<T, VV, true>, grid, dim3(kThreads), 0, stream, a, tb, hb);  \
        else                                                                     \
            return launch_early(rope_kernel<T, VV, false>, grid, dim3(kThreads), 0, stream, a, tb, hb); \
    } while (0)
    if (a.f32 && vec) CSA_ROPE(float, 4);
    if (a.f32) CSA_ROPE(float, 1);
    if (vec) CSA_ROPE(__nv_bfloat16, 8);
    CSA_ROPE(__nv_bfloat16, 1);
#undef CSA_ROPE
}

cudaError_t launch_cache_append(const AppendArgs &a, cudaStream_t stream) {
    const int es = a.f32 ? 4 : 2;
    const bool vec = aligned(a.rows, a.row_stride * es) && aligned(a.cache, a.D * 2) &&
                     a.D % 8 == 0 && a.off % 8 == 0 && a.n % 16 == 0;
    const int units = a.D / (vec ? 8 : 1);
    int sms;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    // rows per block: kPieces units a thread, fewer while that leaves an SM
    // with less than two blocks
    int rows = max(1, kPieces * kThreads / max(units, 1));
    rows = min(rows, max(1, a.T / (2 * sms)));
    int tb = min(rows, kMaxRows);
    if (a.n > 0) tb = max(1, min(tb, kTable / (a.n / 2)));
    const dim3 grid(blocks(a.T, tb));
#define CSA_APPEND(T, VV)                                                          \
    do {                                                                           \
        if (a.half)                                                                \
            return launch_early(cache_append_kernel<T, VV, true>, grid, dim3(kThreads), 0, stream, a, tb); \
        else                                                                       \
            return launch_early(cache_append_kernel<T, VV, false>, grid, dim3(kThreads), 0, stream, a, tb); \
    } while (0)
    if (a.f32 && vec) CSA_APPEND(float, 8);
    if (a.f32) CSA_APPEND(float, 1);
    if (vec) CSA_APPEND(__nv_bfloat16, 8);
    CSA_APPEND(__nv_bfloat16, 1);
#undef CSA_APPEND
}

}  // namespace csa
