// Lightning-indexer score + causal top-k for new tokens of sequences whose
// compressed indexer rows lie in a paged cache (sm_103a).
//
//     s(t, j) = sum_h w[t,h] * max(0, q[t,h,:] . k[j,:])
// over the compressed rows j < floor((pos_t + 1) / cmp_ratio) of t's sequence;
// the topk highest, ties to the lower row, in ascending order.
#include "common.cuh"
#include "internal.h"
#include "paged.h"

namespace csa {

namespace {

constexpr int kScoreRows = 128;
constexpr int kSelThreads = 1024;

// Visible rows of token t and its sequence (-1: none).
__device__ __forceinline__ int32_t visible_rows(const IndexerPagedArgs &a, int32_t t, int32_t *seq,
                                                bool report) {
    const int32_t pos = __ldg(a.q_pos + t);
    const int32_t b = paged_seq(a.q_seq, a.batch, t, pos);
    *seq = b < 0 ? -1 : b;
    if (b < 0) {
        if (b == -2 && report) report_error(a.err, kErrCheck, kKerIndexerPaged, 1);
        return 0;
    }
    const int32_t n = (int32_t)(((int64_t)pos + 1) / a.cmp_ratio);
    if (n > a.max_rows) {
        if (report) report_error(a.err, kErrCheck, kKerIndexerPaged, 2);
        return a.max_rows;
    }
    return n;
}

template <int DI>
__global__ void __launch_bounds__(kScoreRows) indexer_paged_score_kernel(IndexerPagedArgs a) {
    __shared__ float q[64][DI];
    __shared__ float w[64];
    const int32_t t = blockIdx.y;
    int32_t seq;
    const int32_t n = visible_rows(a, t, &seq, false);
    const int32_t j = blockIdx.x * kScoreRows + threadIdx.x;
    if ((int64_t)blockIdx.x * kScoreRows >= n || (n <= a.topk && !a.topk_val)) return;
    for (int i = threadIdx.x; i < a.Hi * DI; i += kScoreRows)
        q[i / DI][i % DI] = (float)a.q[(int64_t)t * a.Hi * DI + i];
    for (int i = threadIdx.x; i < a.Hi; i += kScoreRows) w[i] = a.w[(int64_t)t * a.Hi + i];
    __syncthreads();
    if (j >= n) return;
    const int64_t row = paged_row(a.k, seq, j);
    float s = -INFINITY;
    if (row < 0) {
        report_error(a.err, kErrCheck, kKerIndexerPaged, 3);
    } else {
        const __nv_bfloat16 *k = a.k.base + row * DI;
        s = 0.0f;
        for (int h = 0; h < a.Hi; ++h) {
            float d = 0.0f;
            for (int e = 0; e < DI; ++e) d = fmaf(q[h][e], (float)k[e], d);
            s = fmaf(w[h], fmaxf(d, 0.0f), s);
        }
    }
    a.scores[t * a.row_pad + j] = s;
}

// One block per token: radix select on order-preserving keys.
__global__ void __launch_bounds__(kSelThreads) indexer_paged_select_kernel(IndexerPagedArgs a) {
    __shared__ int32_t hist[256];
    __shared__ int32_t scan[kSelThreads / 32 + 1];
    __shared__ uint32_t range[2];
    __shared__ int32_t pick[2];
    const int32_t t = blockIdx.x, K = a.topk, tid = threadIdx.x;
    int32_t seq;
    const int32_t n = visible_rows(a, t, &seq, tid == 0);
    const float *sc = a.scores + t * a.row_pad;
    int32_t *idx = a.topk_idx + (int64_t)t * K;
    float *val = a.topk_val ? a.topk_val + (int64_t)t * K : nullptr;
    if (n <= K) {
        for (int32_t i = tid; i < K; i += kSelThreads) {
            idx[i] = i < n ? i : -1;
            if (val) val[i] = i < n ? sc[i] : -INFINITY;
        }
        return;
    }
    if (tid == 0) {
        range[0] = 0xffffffffu;
        range[1] = 0u;
    }
    __syncthreads();
    uint32_t lo = 0xffffffffu, hi = 0u;
    for (int32_t i = tid; i < n; i += kSelThreads) {
        const uint32_t k = float_key(sc[i]);
        lo = min(lo, k);
        hi = max(hi, k);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if ((tid & 31) == 0) {
        atomicMin(&range[0], lo);
        atomicMax(&range[1], hi);
    }
    __syncthreads();
    lo = range[0];
    hi = range[1];
    const int free_bits = lo == hi ? 0 : 32 - __clz((int)(lo ^ hi));
    uint32_t mask = free_bits == 32 ? 0u : ~((1u << free_bits) - 1u);
    uint32_t prefix = lo & mask;
    int32_t left = K;  // still to take from the bucket
    for (int top = free_bits; top > 0; top -= 8) {
        const int shift = max(top - 8, 0);
        const uint32_t dmask = (1u << (top - shift)) - 1u;
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int32_t i = tid; i < n; i += kSelThreads) {
            const uint32_t k = float_key(sc[i]);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & dmask], 1);
        }
        __syncthreads();
        int32_t total;
        const int32_t c = tid < 256 ? hist[255 - tid] : 0;
        const int32_t above = block_exclusive_scan<kSelThreads>(c, scan, &total);
        if (tid < 256 && above < left && left <= above + c) {
            pick[0] = 255 - tid;
            pick[1] = above;
        }
        __syncthreads();
        prefix |= (uint32_t)pick[0] << shift;
        mask |= dmask << shift;
        left -= pick[1];
        __syncthreads();
    }
    int32_t out = 0, eq_seen = 0;
    for (int32_t i0 = 0; i0 < n; i0 += kSelThreads) {
        const int32_t i = i0 + tid;
        const uint32_t k = i < n ? float_key(sc[i]) & mask : 0u;
        const bool gt = i < n && k > prefix, eq = i < n && k == prefix;
        int32_t eqs, taken;
        const int32_t eb = block_exclusive_scan<kSelThreads>(eq ? 1 : 0, scan, &eqs);
        const bool take = gt || (eq && eq_seen + eb < left);
        const int32_t at = block_exclusive_scan<kSelThreads>(take ? 1 : 0, scan, &taken);
        if (take) {
            idx[out + at] = i;
            if (val) val[out + at] = sc[i];
        }
        out += taken;
        eq_seen += eqs;
    }
}

}  // namespace

size_t indexer_paged_workspace_bytes(int32_t T, int64_t max_rows) {
    return (size_t)T * (size_t)((max_rows + 63) / 64 * 64) * sizeof(float);
}

cudaError_t launch_indexer_topk_paged(IndexerPagedArgs a, cudaStream_t stream) {
    a.row_pad = ((int64_t)a.max_rows + 63) / 64 * 64;
    const dim3 grid((a.max_rows + kScoreRows - 1) / kScoreRows, a.T);
    if (grid.x > 0) {
        if (a.Di == 128)
            indexer_paged_score_kernel<128><<<grid, kScoreRows, 0, stream>>>(a);
        else
            indexer_paged_score_kernel<64><<<grid, kScoreRows, 0, stream>>>(a);
    }
    indexer_paged_select_kernel<<<a.T, kSelThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace csa
