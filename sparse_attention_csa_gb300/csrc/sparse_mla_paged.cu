// Sparse MLA attention of new tokens over paged caches (sm_103a): the keys of
// token t are the window rows of its sequence in the original-KV cache and the
// listed (or every visible) rows of the compressed cache.
//
//     l_i = scale q.kv_i ; Z = sum e^(l_i - m) + e^(sink - m)
//     out = sum e^(l_i - m) kv_i / Z ; lse = m + ln Z
//
// Work split. A token's keys form tiles of 64 slots; the tiles of all tokens,
// one after the other, are dealt to the CTAs in equal runs, so a long row is
// spread over many CTAs and short ones share one, whatever the lengths are. A
// run covers the end of one token, whole tokens, and the start of one more;
// whole tokens are finished in place, and a CTA's one or two pieces of tokens
// go to its two slots of the workspace (fp32 sums with their running maximum),
// which the CTA that holds a token's first tile describes and a second kernel
// joins. The split depends on the sizes alone, so results repeat bit by bit.
#include "common.cuh"
#include "internal.h"
#include "paged.h"

namespace csa {

namespace {

constexpr int kTile = 64;
constexpr int kMaxGrid = 160;  // CTAs of the persistent grid (sizes the workspace)
constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Join {
    int32_t t, first, last, pad;  // token split over CTAs first..last (t < 0: none)
};

// Workspace: Join [kMaxGrid], then m and l [2 kMaxGrid][H], then the sums
// [2 kMaxGrid][H][512].
struct Space {
    Join *join;
    float *m, *l, *o;
    __host__ __device__ Space(void *p, int32_t H) {
        join = static_cast<Join *>(p);
        m = reinterpret_cast<float *>(join + kMaxGrid);
        l = m + 2 * kMaxGrid * H;
        o = l + 2 * kMaxGrid * H;
    }
};

// Key slots of a token, from its position alone.
struct Keys {
    int32_t seq, win_start, n_win, vis, n_cmp;
    __device__ __forceinline__ int32_t slots() const { return n_win + n_cmp; }
    __device__ __forceinline__ int32_t tiles() const {  // a token without keys has one, empty
        const int32_t n = (int32_t)(((int64_t)n_win + n_cmp + kTile - 1) / kTile);
        return n > 0 ? n : 1;
    }
};

__device__ __forceinline__ Keys token_keys(const MlaPagedArgs &a, int32_t t, bool report) {
    Keys k = {-1, 0, 0, 0, 0};
    const int32_t pos = __ldg(a.q_pos + t);
    const int32_t b = paged_seq(a.q_seq, a.batch, t, pos);
    if (b < 0) {
        if (b == -2 && report) report_error(a.err, kErrCheck, kKerMlaPaged, 1);
        return k;
    }
    k.seq = b;
    k.win_start = max(pos - a.window + 1, 0);
    k.n_win = pos - k.win_start + 1;
    if (a.cmp.base) {
        const int64_t cap = (int64_t)a.cmp.max_pages * a.cmp.page_size;
        int64_t vis = ((int64_t)pos + 1) / a.cmp_ratio;
        if (vis > cap) {
            if (report) report_error(a.err, kErrCheck, kKerMlaPaged, 2);
            vis = cap;
        }
        k.vis = (int32_t)vis;
        k.n_cmp = a.idx ? (k.vis > 0 ? a.topk : 0) : k.vis;
    }
    return k;
}

// Pool row of key slot i of token t (nullptr: no key there).
__device__ __forceinline__ const __nv_bfloat16 *key_row(const MlaPagedArgs &a, const Keys &k,
                                                        int32_t t, int32_t i) {
    if (i >= k.slots()) return nullptr;
    const bool win = i < k.n_win;
    int32_t r = win ? k.win_start + i : i - k.n_win;
    if (!win && a.idx) {
        r = __ldg(a.idx + (int64_t)t * a.topk + r);
        if (r < 0 || r >= k.vis) return nullptr;
    }
    const PagedRows &p = win ? a.ori : a.cmp;
    const int64_t row = paged_row(p, k.seq, r);
    if (row < 0) {
        report_error(a.err, kErrCheck, kKerMlaPaged, 3);
        return nullptr;
    }
    return p.base + row * 512;
}

__global__ void __launch_bounds__(kThreads) sparse_mla_paged_kernel(MlaPagedArgs a) {
    __shared__ const __nv_bfloat16 *rows[kTile];
    __shared__ float p[64][kTile + 1];
    __shared__ float m_s[64], l_s[64], al_s[64];
    __shared__ int64_t sums[2];
    const int tid = threadIdx.x;
    const Space ws(a.workspace, a.H);
    const int32_t c = blockIdx.x;
    if (tid == 0) {
        int64_t N = 0;
        for (int32_t t = 0; t < a.T; ++t) N += token_keys(a, t, c == 0).tiles();
        sums[0] = N;
        ws.join[c] = {-1, 0, 0, 0};
    }
    __syncthreads();
    const int64_t N = sums[0], G = min((int64_t)gridDim.x, N);  // every run holds a tile
    if (c >= G) return;
    const int64_t s = c * N / G, e = (c + 1) * N / G;
    int64_t base = 0;
    for (int32_t t = 0; t < a.T && base < e; ++t) {
        const Keys k = token_keys(a, t, false);
        const int32_t nt = k.tiles();
        const int64_t b0 = base;
        base += nt;
        if (base <= s) continue;
        const int32_t j0 = (int32_t)max(s - b0, (int64_t)0), j1 = (int32_t)min(e - b0, (int64_t)nt);
        const bool whole = j0 == 0 && j1 == nt;
        float o[64][2];
        for (int h = 0; h < 64; ++h) o[h][0] = o[h][1] = 0.0f;
        __syncthreads();
        if (tid < 64) {
            m_s[tid] = -INFINITY;
            l_s[tid] = 0.0f;
        }
        for (int32_t j = j0; j < j1; ++j) {
            __syncthreads();
            if (tid < kTile) rows[tid] = key_row(a, k, t, j * kTile + tid);
            __syncthreads();
            for (int i = tid; i < a.H * kTile; i += kThreads) {
                const int h = i / kTile, x = i % kTile;
                float d = -INFINITY;
                if (rows[x]) {
                    d = 0.0f;
                    const __nv_bfloat16 *q = a.q + ((int64_t)t * a.H + h) * 512;
                    for (int u = 0; u < 512; ++u) d = fmaf((float)q[u], (float)rows[x][u], d);
                    d *= a.softmax_scale * kLog2e;
                }
                p[h][x] = d;
            }
            __syncthreads();
            if (tid < a.H) {
                float m = m_s[tid];
                for (int x = 0; x < kTile; ++x) m = fmaxf(m, p[tid][x]);
                const float al = m == -INFINITY ? 1.0f : exp2f(m_s[tid] - m);
                float l = l_s[tid] * al;
                for (int x = 0; x < kTile; ++x) {
                    const float v = m == -INFINITY ? 0.0f : exp2f(p[tid][x] - m);
                    p[tid][x] = v;
                    l += v;
                }
                m_s[tid] = m;
                l_s[tid] = l;
                al_s[tid] = al;
            }
            __syncthreads();
            for (int h = 0; h < a.H; ++h)
                for (int u = 0; u < 2; ++u) {
                    float acc = o[h][u] * al_s[h];
                    for (int x = 0; x < kTile; ++x)
                        if (rows[x]) acc = fmaf(p[h][x], (float)rows[x][2 * tid + u], acc);
                    o[h][u] = acc;
                }
        }
        __syncthreads();
        if (whole) {
            for (int h = 0; h < a.H; ++h) {
                const float sk = k.seq >= 0 && a.sinks ? a.sinks[h] * kLog2e : -INFINITY;
                const float M = fmaxf(m_s[h], sk);
                const float f = m_s[h] == -INFINITY ? 0.0f : exp2f(m_s[h] - M);
                const float Z = l_s[h] * f + (sk == -INFINITY ? 0.0f : exp2f(sk - M));
                for (int u = 0; u < 2; ++u)
                    a.out[((int64_t)t * a.H + h) * 512 + 2 * tid + u] =
                        __float2bfloat16_rn(Z > 0.0f ? o[h][u] * f / Z : 0.0f);
                if (tid == 0 && a.lse) a.lse[(int64_t)t * a.H + h] = (M + log2f(Z)) * kLn2;
            }
        } else {
            const int32_t slot = 2 * c + (j0 == 0 ? 1 : 0);
            if (j0 == 0 && tid == 0)
                ws.join[c] = {t, c, (int32_t)(((b0 + nt) * G - 1) / N), k.seq};
            for (int h = 0; h < a.H; ++h) {
                for (int u = 0; u < 2; ++u)
                    ws.o[((int64_t)slot * a.H + h) * 512 + 2 * tid + u] = o[h][u];
                if (tid == 0) {
                    ws.m[slot * a.H + h] = m_s[h];
                    ws.l[slot * a.H + h] = l_s[h];
                }
            }
        }
    }
}

// Block (c, y): heads 8y .. 8y + 7 of the token whose first tile CTA c held
// and that other CTAs went on with; one warp per head, 16 dims per lane.
__global__ void __launch_bounds__(256) sparse_mla_paged_join_kernel(MlaPagedArgs a) {
    const Space ws(a.workspace, a.H);
    const Join jn = ws.join[blockIdx.x];
    if (jn.t < 0) return;
    const int h = 8 * blockIdx.y + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (h >= a.H) return;
    const float sk = a.sinks ? a.sinks[h] * kLog2e : -INFINITY;
    auto slot = [&](int32_t c) { return c == jn.first ? 2 * c + 1 : 2 * c; };
    float M = sk;
    for (int32_t c = jn.first; c <= jn.last; ++c) M = fmaxf(M, ws.m[slot(c) * a.H + h]);
    float Z = sk == -INFINITY ? 0.0f : exp2f(sk - M);
    float o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.0f;
    for (int32_t c = jn.first; c <= jn.last; ++c) {
        const int32_t s = slot(c);
        const float m = ws.m[s * a.H + h];
        const float f = m == -INFINITY ? 0.0f : exp2f(m - M);
        Z = fmaf(ws.l[s * a.H + h], f, Z);
        const float4 *src = reinterpret_cast<const float4 *>(ws.o + ((int64_t)s * a.H + h) * 512);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = src[32 * i + lane];
            o[4 * i] = fmaf(v.x, f, o[4 * i]);
            o[4 * i + 1] = fmaf(v.y, f, o[4 * i + 1]);
            o[4 * i + 2] = fmaf(v.z, f, o[4 * i + 2]);
            o[4 * i + 3] = fmaf(v.w, f, o[4 * i + 3]);
        }
    }
    const float r = Z > 0.0f ? 1.0f / Z : 0.0f;
    __nv_bfloat16 *out = a.out + ((int64_t)jn.t * a.H + h) * 512;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(o[4 * i] * r, o[4 * i + 1] * r);
        const __nv_bfloat162 y = __floats2bfloat162_rn(o[4 * i + 2] * r, o[4 * i + 3] * r);
        reinterpret_cast<uint2 *>(out)[32 * i + lane] =
            make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    }
    if (lane == 0 && a.lse)
        a.lse[(int64_t)jn.t * a.H + h] = (M + log2f(Z)) * kLn2;
}

}  // namespace

size_t mla_paged_workspace_bytes(int32_t T, int32_t H) {
    if (T <= 0) return 0;
    return kMaxGrid * sizeof(Join) + (size_t)2 * kMaxGrid * H * (512 + 2) * sizeof(float);
}

cudaError_t launch_sparse_mla_paged(MlaPagedArgs a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int grid = min(sms, kMaxGrid);
    sparse_mla_paged_kernel<<<grid, kThreads, 0, stream>>>(a);
    sparse_mla_paged_join_kernel<<<dim3(grid, (a.H + 7) / 8), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace csa
