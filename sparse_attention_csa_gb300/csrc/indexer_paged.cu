// Lightning-indexer score + causal top-k for new tokens of sequences whose
// compressed indexer rows lie in a paged cache (sm_103a, tcgen05, cp.async,
// thread-block clusters).
//
//     s(t, j) = sum_h w[t,h] * max(0, q[t,h,:] . k[j,:])
// over the compressed rows j < floor((pos_t + 1) / cmp_ratio) of t's sequence;
// the topk highest, ties to the lower row, in ascending order.
//
// Two kernels.
//
// Scores. Every row is read once for its token (256 bytes for 2 x 64 x 128
// operations: bound by HBM). The 128-row tiles of all tokens that need scoring
// are dealt to the CTAs in equal runs. A tile is the MMA's M side, the heads
// its N side: S[j, h] = k[j,:] . q[h,:], so that with one TMEM lane a row the
// sum over heads stays inside a thread. Five stages of 32 KB (eight of 16 KB
// with 64-wide rows) keep 128 KB or more on their way; four loader warps
// gather, one thread issues, four warps reduce. A token that sees at most topk
// rows selects all of them and is not scored unless its values are asked for.
//
// Selection. A cluster of up to eight CTAs takes a token, each an even share
// of its rows, held in registers. One histogram of 2048 linear bins between
// the smallest and the largest score (equal scores share a bin, larger ones
// never fall lower) nearly always leaves a handful of candidates in the bin of
// the topk-th; they are ranked directly. More than kCand of them (outliers,
// equal scores, infinities) go through radix passes over that bin's keys. The
// rows are emitted in order by counts over lanes, warps and CTAs. Bound by the
// latency of its steps: 2 MB read.
//
// The number of CTAs a token, whether they hold their rows, and the workspace
// follow from what the page table can hold, not from what a token sees: a table
// much wider than its sequences costs CTAs without rows and, past 65536 rows,
// sweeps that read the scores again (64 tokens of up to 16384 rows: 39.8 us
// with a table that fits, 41.8 with one of 32768 rows, 62 with 65600 or more).
//
// Both together: one token over 32768 rows 14.4 us; 64 tokens over 0.57 million
// rows, 146 MB, 39.8 us, the scores alone at 4.5 TB/s under a profiler.
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "tc_ptx.cuh"

namespace csa {

namespace {

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
    const int32_t n = (int32_t)(((uint32_t)pos + 1u) / (uint32_t)a.cmp_ratio);
    if (n > a.max_rows) {
        if (report) report_error(a.err, kErrCheck, kKerIndexerPaged, 2);
        return a.max_rows;
    }
    return n;
}

// ------------------------------------------------------------------- scores
constexpr int kTileRows = 128;
constexpr int kThreads = 288;  // 4 epilogue warps, 4 loader warps, 1 MMA warp
constexpr int kLoaders = 128;
constexpr int kMmaWarp = 8;
constexpr int kPieces = 64;    // tokens of a run described in shared memory at a time
constexpr int kAcc = 4;        // tensor-memory accumulators of 64 columns

struct Piece {
    int32_t t, j0, j1, n, seq;  // tiles [j0, j1) of token t, which sees n rows
};

template <int DI>
struct Score {
    static constexpr int kChunks = DI / 64;                  // 128-byte chunks of a row
    static constexpr uint32_t kStage = kTileRows * DI * 2;
    static constexpr int kStages = DI == 128 ? 5 : 8;
    static constexpr uint32_t kQ = 64 * DI * 2;
    static constexpr uint32_t kOffQ = 0;                     // two tokens' heads
    static constexpr uint32_t kOffK = 2 * kQ;
    static constexpr uint32_t kOffMisc = kOffK + kStages * kStage;
    struct Misc {
        uint64_t q_full[2], q_empty[2];
        uint64_t k_full[kStages], k_empty[kStages];
        uint64_t acc_full[kAcc], acc_empty[kAcc];
        uint64_t drain;
        int64_t run_base, done;
        int32_t run_t, n_pieces;
        uint32_t tmem_base;
        int32_t abort;
        int32_t scan[kThreads / 32 + 1];
        uint32_t present[kStages][4];  // a stage's rows whose page exists
        Piece piece[kPieces];
        alignas(16) float w[2][64];
    };
    static constexpr size_t kSmem = kOffMisc + sizeof(Misc) + 1024;
    static_assert(kSmem <= 232448, "shared memory budget");
};

template <int DI>
__global__ void __launch_bounds__(kThreads, 1)
indexer_paged_score_kernel(const __grid_constant__ IndexerPagedArgs a) {
    using S = Score<DI>;
    using Misc = typename S::Misc;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc *ms = reinterpret_cast<Misc *>(smem + S::kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PipeWaits<Misc, kKerIndexerPaged> cx{ms, a.err, a.wait_ns};
    const int32_t c = blockIdx.x;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&ms->q_full[i], kLoaders);
            tc::mbar_init(&ms->q_empty[i], 1 + 128);
        }
        for (int i = 0; i < S::kStages; ++i) {
            tc::mbar_init(&ms->k_full[i], kLoaders + 4);
            tc::mbar_init(&ms->k_empty[i], 1 + 128);
        }
        for (int i = 0; i < kAcc; ++i) {
            tc::mbar_init(&ms->acc_full[i], 1);
            tc::mbar_init(&ms->acc_empty[i], 128);
        }
        tc::mbar_init(&ms->drain, 1);
        ms->abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&ms->tmem_base, 64 * kAcc);
        tc::tmem_relinquish();
    }
    // heads past Hi: zero rows of both q buffers, never written again
    for (int i = tid; i < 2 * (64 - a.Hi) * (DI / 8); i += kThreads) {
        const int buf = i / ((64 - a.Hi) * (DI / 8)), r = i - buf * (64 - a.Hi) * (DI / 8);
        const int h = a.Hi + r / (DI / 8), u = r % (DI / 8);
        *reinterpret_cast<uint4 *>(smem + S::kOffQ + buf * S::kQ + (u >> 3) * 8192 + h * 128 +
                                   (u & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
    if (tid < 128) ms->w[tid >> 6][tid & 63] = 0.0f;
    // everything above is local: wait for the kernels before this one
    grid_dependency_wait();
    launch_dependents();
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();

    // ------------------------------------------------ this CTA's run of tiles
    auto tiles_of = [&](int32_t t, int32_t *n, int32_t *seq) -> int32_t {
        *n = visible_rows(a, t, seq, false);
        return *n > a.topk || a.topk_val ? (*n + kTileRows - 1) / kTileRows : 0;
    };
    const bool one_scan = a.T <= kThreads;
    int32_t n = 0, seq = -1, nt = 0, total = 0;
    int64_t N = 0, b = 0;
    for (int32_t t0 = 0; t0 < a.T; t0 += kThreads) {
        const int32_t t = t0 + tid;
        nt = t < a.T ? tiles_of(t, &n, &seq) : 0;
        b = block_exclusive_scan<kThreads>(nt, ms->scan, &total);
        N += total;
    }
    tc::tc_fence_after();
    const uint32_t tmem = ms->tmem_base;
    const int64_t per = div64(N + gridDim.x - 1, gridDim.x);
    const int64_t s = min(c * per, N), e = min(s + per, N);
    if (s == e) {  // no run left for this CTA
        __syncthreads();
        if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 64 * kAcc);
        return;
    }
    if (one_scan) {
        if (b <= s && s < b + nt) ms->run_t = tid;
    } else {  // the token holding tile s
        int64_t base = 0;
        for (int32_t t0 = 0; t0 < a.T && base <= s; t0 += kThreads) {
            const int32_t t = t0 + tid;
            const int32_t k = t < a.T ? tiles_of(t, &n, &seq) : 0;
            const int64_t bt = base + block_exclusive_scan<kThreads>(k, ms->scan, &total);
            if (bt <= s && s < bt + k) {
                ms->run_t = t;
                ms->run_base = bt;
            }
            base += total;
        }
    }
    __syncthreads();

    uint32_t g = 0, np = 0;  // tiles and tokens so far, kept by every role
    bool issued = false;
    int64_t done = s;
    while (done < e) {
        // ------------------------------------------------- a batch of tokens
        const int32_t t_first = ms->run_t;
        int32_t t = tid;
        int x = tid - t_first;  // place in the batch
        if (!one_scan) {
            const int64_t base = ms->run_base;
            t = t_first + tid;
            x = tid;
            nt = tid < kPieces && t < a.T ? tiles_of(t, &n, &seq) : 0;
            b = base + block_exclusive_scan<kThreads>(nt, ms->scan, &total);
        }
        if (x >= 0 && x < kPieces && t < a.T && b < e) {  // a token without tiles has an empty piece
            ms->piece[x] = {t, (int32_t)max(s - b, (int64_t)0), (int32_t)min(e - b, (int64_t)nt), n, seq};
            if (x == kPieces - 1 || t + 1 == a.T || b + nt >= e) {
                ms->n_pieces = x + 1;
                ms->done = min(e, b + nt);
            }
        }
        __syncthreads();
        done = ms->done;
        const int32_t n_pieces = ms->n_pieces;
        if (tid == 0) {
            ms->run_t = t_first + kPieces;
            if (!one_scan) ms->run_base += total;
        }

        if (warp == kMmaWarp) {
            // ===================================================== MMA warp
            if (lane == 0) {
                constexpr uint32_t id = tc::idesc_bf16(128, 64, false, false);
                const uint64_t da = tc::smem_desc(tc::smem_u32(smem + S::kOffK), 16, 1024);
                const uint64_t db = tc::smem_desc(tc::smem_u32(smem + S::kOffQ), 16, 1024);
                bool ok = true;
                for (int32_t i = 0; i < n_pieces && ok; ++i) {
                    const int32_t j0 = ms->piece[i].j0, j1 = ms->piece[i].j1;
                    if (j0 >= j1) continue;
                    ok = cx.wait(&ms->q_full[np & 1], (np >> 1) & 1, 20);
                    for (int32_t j = j0; j < j1 && ok; ++j, ++g) {
                        const uint32_t st = g % S::kStages, acc = g % kAcc;
                        ok = cx.wait(&ms->k_full[st], (g / S::kStages) & 1, 21) &&
                             cx.wait(&ms->acc_empty[acc], ((g / kAcc) & 1) ^ 1, 22);
                        if (!ok) break;
                        tc::fence_proxy_async_smem();  // cp.async wrote through the generic proxy
                        tc::tc_fence_after();
#pragma unroll
                        for (int ch = 0; ch < S::kChunks; ++ch)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc::mma_bf16(tmem + 64 * acc,
                                             tc::desc_add(da, st * S::kStage + ch * 16384 + kk * 32),
                                             tc::desc_add(db, (np & 1) * S::kQ + ch * 8192 + kk * 32), id,
                                             (ch | kk) != 0);
                        issued = true;
                        tc::mma_commit(&ms->k_empty[st]);
                        tc::mma_commit(&ms->acc_full[acc]);
                    }
                    if (ok) tc::mma_commit(&ms->q_empty[np & 1]);
                    ++np;
                }
            }
            __syncwarp();
        } else if (warp >= 4) {
            // ================================================= loader warps
            // Warp w: rows 32 w .. 32 w + 31 of every tile, looked up one a
            // lane, a tile ahead.
            const int w = warp - 4, li = tid - 128;
            bool ok = true;
            for (int32_t i = 0; i < n_pieces && ok; ++i) {
                const Piece p = ms->piece[i];
                if (p.j0 >= p.j1) continue;
                auto page_of = [&](int32_t j, int32_t *in) -> int32_t {
                    const int64_t r = (int64_t)j * kTileRows + 32 * w + lane;
                    *in = -1;
                    if (j >= p.j1 || r >= p.n) return -1;
                    const uint32_t pg = (uint32_t)r / (uint32_t)a.k.page_size;  // in the table: n <= max_rows
                    *in = (int32_t)r - (int32_t)pg * a.k.page_size;
                    return __ldg(a.k.pages + (int64_t)p.seq * a.k.max_pages + pg);
                };
                int32_t in, in_next;
                int32_t page = page_of(p.j0, &in), page_next = page_of(p.j0 + 1, &in_next);
                ok = __all_sync(0xffffffffu, cx.wait(&ms->q_empty[np & 1], ((np >> 1) & 1) ^ 1, 40));
                if (!ok) break;
                const __nv_bfloat16 *q = a.q + (int64_t)p.t * a.Hi * DI;
                for (int u = li; u < a.Hi * (DI / 8); u += kLoaders) {
                    const int h = u / (DI / 8), y = u % (DI / 8);
                    cp_async16(tc::smem_u32(smem + S::kOffQ) + (np & 1) * S::kQ + (y >> 3) * 8192 + h * 128 +
                                   (((y & 7) ^ (h & 7)) << 4),
                               q + (int64_t)u * 8, 16);
                }
                if (li < a.Hi)  // weights past Hi stay zero
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                                     tc::smem_u32(&ms->w[np & 1][li])),
                                 "l"(a.w + (int64_t)p.t * a.Hi + li)
                                 : "memory");
                cp_async_arrive(&ms->q_full[np & 1]);
                ++np;
                for (int32_t j = p.j0; j < p.j1; ++j, ++g) {
                    const uint32_t st = g % S::kStages;
                    const __nv_bfloat16 *mine = nullptr;
                    if (in >= 0) {
                        if ((uint32_t)page < (uint32_t)a.k.num_pages)
                            mine = a.k.base + ((int64_t)page * a.k.page_size + in) * DI;
                        else
                            report_error(a.err, kErrCheck, kKerIndexerPaged, 3);
                    }
                    const uint32_t m = __ballot_sync(0xffffffffu, mine != nullptr);
                    page = page_next;
                    in = in_next;
                    page_next = page_of(j + 2, &in_next);
                    ok = __all_sync(0xffffffffu, cx.wait(&ms->k_empty[st], ((g / S::kStages) & 1) ^ 1, 41));
                    if (!ok) break;
                    // 512 bytes an instruction: two rows (four of 64 dims)
                    constexpr int kLanes = DI / 8, kRows = 32 / kLanes;
                    const int y = lane % kLanes, sub = lane / kLanes;
                    const uint32_t base = tc::smem_u32(smem + S::kOffK) + st * S::kStage + (y >> 3) * 16384;
#pragma unroll
                    for (int r = 0; r < 32 / kRows; ++r) {
                        const int row = kRows * r + sub;
                        const __nv_bfloat16 *src = reinterpret_cast<const __nv_bfloat16 *>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), row));
                        cp_async16(base + (32 * w + row) * 128 + (((y & 7) ^ (row & 7)) << 4),
                                   (src ? src : a.q) + y * 8, src ? 16u : 0u);
                    }
                    cp_async_arrive(&ms->k_full[st]);
                    if (lane == 0) {
                        ms->present[st][w] = m;
                        tc::mbar_arrive(&ms->k_full[st]);
                    }
                }
            }
        } else {
            // =============================================== epilogue warps
            // Every wait's result is the warp's, not a lane's: what follows is
            // collective, and lanes that gave up must not part from the others.
            const uint32_t lane_addr = tmem + ((uint32_t)(32 * warp) << 16);
            bool ok = true;
            for (int32_t i = 0; i < n_pieces && ok; ++i) {
                const Piece p = ms->piece[i];
                if (p.j0 >= p.j1) continue;
                ok = __all_sync(0xffffffffu, cx.wait(&ms->q_full[np & 1], (np >> 1) & 1, 30));
                if (!ok) break;
                const float4 *w4 = reinterpret_cast<const float4 *>(ms->w[np & 1]);
                float *out = a.scores + (int64_t)p.t * a.row_pad;
                for (int32_t j = p.j0; j < p.j1; ++j, ++g) {
                    const uint32_t st = g % S::kStages, acc = g % kAcc;
                    ok = __all_sync(0xffffffffu, cx.wait(&ms->k_full[st], (g / S::kStages) & 1, 31) &&
                                                     cx.wait(&ms->acc_full[acc], (g / kAcc) & 1, 32));
                    if (!ok) break;
                    tc::tc_fence_after();
                    const bool there = (ms->present[st][warp] >> lane) & 1u;
                    tc::mbar_arrive(&ms->k_empty[st]);
                    float sum[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        float v[32];
                        tc::tmem_ld32(lane_addr + 64 * acc + 32 * hh, v);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const float4 w = w4[8 * hh + y];
                            sum[0] = fmaf(w.x, fmaxf(v[4 * y], 0.0f), sum[0]);
                            sum[1] = fmaf(w.y, fmaxf(v[4 * y + 1], 0.0f), sum[1]);
                            sum[0] = fmaf(w.z, fmaxf(v[4 * y + 2], 0.0f), sum[0]);
                            sum[1] = fmaf(w.w, fmaxf(v[4 * y + 3], 0.0f), sum[1]);
                        }
                    }
                    tc::tc_fence_before();
                    tc::mbar_arrive(&ms->acc_empty[acc]);
                    const int64_t r = (int64_t)j * kTileRows + 32 * warp + lane;
                    if (r < p.n) out[r] = there ? (sum[0] + sum[1]) + 0.0f : -INFINITY;  // no -0
                }
                if (ok) tc::mbar_arrive(&ms->q_empty[np & 1]);
                ++np;
            }
        }
        __syncthreads();
        if (cx.aborted()) break;
    }

    // ------------------------------------------------------------- teardown
    if (warp >= 4 && warp < kMmaWarp) asm volatile("cp.async.wait_all;" ::: "memory");
    if (tid == 32 * kMmaWarp && issued) {  // no MMA outlives its tensor memory
        tc::mma_commit(&ms->drain);
        if (!tc::mbar_wait(&ms->drain, 0)) cx.fail(24);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 64 * kAcc);
}

// ---------------------------------------------------------------- selection
constexpr int kSelThreads = 512;
constexpr int kQuads = 4;                               // float4 a thread
constexpr int kSelRows = kSelThreads * 4 * kQuads;      // rows a CTA holds in registers
constexpr int kBins = 2048;
constexpr int kCand = 256;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 4 or 16 bytes of CTA `rank`'s shared memory, at this CTA's address p
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(p)), "r"(rank));
    return at;
}
__device__ __forceinline__ uint32_t peer_u32(const void *p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint4 peer_u128(const void *p, uint32_t rank) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(peer_addr(p, rank))
                 : "memory");
    return v;
}

// A score's rank as an unsigned number, from its bits alone (the score kernel
// writes no -0, so equal scores have equal keys). A NaN lies at an end of the
// order, above +inf as the score kernel writes it, and so is the smallest or the
// largest key: there are no bins then. (float_key adds 0 first, and what the
// compiler makes of that ranks a NaN below zero, where linear bins would count
// it among the lowest: more rows written than counted.)
__device__ __forceinline__ uint32_t row_key(float s) {
    const uint32_t u = __float_as_uint(s);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

struct Sel {
    alignas(16) uint32_t hist[kBins];
    uint32_t digit[2][256];
    uint32_t cand[kCand];
    uint32_t all[kCand];
    uint32_t n_cand;
    uint32_t range[2];
    uint32_t counts[2];     // this CTA's rows above the threshold and on it
    uint32_t pick[3];
    int32_t scan[kSelThreads / 32 + 1];
    uint32_t warps[kSelThreads / 32];
};

// C CTAs a token. kHeld: a CTA's share fits its registers; else every sweep
// reads it again.
template <int C, bool kHeld>
__global__ void __launch_bounds__(kSelThreads, 2)
indexer_paged_select_kernel(const __grid_constant__ IndexerPagedArgs a) {
    __shared__ Sel sm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = C > 1 ? cluster_rank() : 0;
    const int32_t t = blockIdx.x / C, K = a.topk;
    auto sync = [&]() {
        if (C > 1) cluster_sync();
        else __syncthreads();
    };
    // one word of every CTA, CTA r's in lane r (`none` in the other lanes)
    auto gather = [&](const uint32_t *p, uint32_t none) -> uint32_t {
        if (lane >= C) return none;
        return C > 1 ? peer_u32(p, lane) : *static_cast<const volatile uint32_t *>(p);
    };
    for (int i = tid; i < kBins; i += kSelThreads) sm.hist[i] = 0;
    if (tid < 256) sm.digit[0][tid] = 0;
    if (tid < 2) sm.counts[tid] = 0;
    if (tid == 0) {
        sm.n_cand = 0;
        sm.range[0] = 0xffffffffu;
        sm.range[1] = 0u;
    }
    grid_dependency_wait();
    launch_dependents();
    int32_t seq;
    const int32_t n = visible_rows(a, t, &seq, tid == 0 && rank == 0);
    const float *sc = a.scores + (int64_t)t * a.row_pad;
    int32_t *idx = a.topk_idx + (int64_t)t * K;
    float *val = a.topk_val ? a.topk_val + (int64_t)t * K : nullptr;
    if (n <= K) {  // every CTA of the cluster alike
        for (int32_t i = rank * kSelThreads + tid; i < K; i += C * kSelThreads) {
            idx[i] = i < n ? i : -1;
            if (val) val[i] = i < n ? sc[i] : -INFINITY;
        }
        return;
    }
    // This CTA's rows [r0, r1), a multiple of 128 apart: chunks of kSelRows, in
    // which a thread holds 4 kQuads consecutive rows (so that one scan over the
    // threads gives every row its place in the output).
    const int32_t share = (int32_t)((((int64_t)n + C - 1) / C + 127) / 128 * 128);
    const int32_t r0 = (int32_t)min((int64_t)rank * share, (int64_t)n);
    const int32_t r1 = (int32_t)min((int64_t)r0 + share, (int64_t)n);
    float4 held[kQuads];
    auto row_at = [&](int32_t c0, int i) { return c0 + 4 * (kQuads * tid + i); };
    auto fetch = [&](int32_t c0) {
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {  // row_pad is a multiple of 64: whole float4 are in bounds
            const int32_t r = row_at(c0, i);
            held[i] = r < r1 ? *reinterpret_cast<const float4 *>(sc + r)
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
    };
    auto each = [&](int32_t c0, auto f) {  // every row of a chunk that exists
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            const int32_t r = row_at(c0, i);
            const float v[4] = {held[i].x, held[i].y, held[i].z, held[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (r + e < r1) f(v[e]);
        }
    };
    auto sweep = [&](auto f) {
        if (kHeld) {
            each(r0, f);
        } else {
            for (int32_t c0 = r0; c0 < r1; c0 += kSelRows) {
                fetch(c0);
                each(c0, f);
            }
        }
    };
    if (kHeld) fetch(r0);
    __syncthreads();
    // ---- smallest and largest key
    {
        uint32_t lo = 0xffffffffu, hi = 0u;
        sweep([&](float s) {
            const uint32_t k = row_key(s);
            lo = min(lo, k);
            hi = max(hi, k);
        });
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
            atomicMin(&sm.range[0], lo);
            atomicMax(&sm.range[1], hi);
        }
    }
    sync();
    const uint32_t lo = __reduce_min_sync(0xffffffffu, gather(&sm.range[0], 0xffffffffu));
    const uint32_t hi = __reduce_max_sync(0xffffffffu, gather(&sm.range[1], 0u));
    auto key_float = [](uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); };
    const float fl = key_float(lo), span = key_float(hi) - fl;
    // no bins without a finite, positive span (a NaN among the scores makes it
    // one): all rows are candidates of bin 0
    const float scale = span > 0.0f && span < INFINITY ? (float)(kBins - 1) / span : 0.0f;
    const bool binned = scale > 0.0f && scale < INFINITY;
    auto bin_of = [&](float s) -> uint32_t {
        return binned ? min((uint32_t)((s - fl) * scale), (uint32_t)(kBins - 1)) : 0u;
    };
    // ---- histogram, and the bin of the K-th largest
    sweep([&](float s) { atomicAdd(&sm.hist[bin_of(s)], 1u); });
    sync();
    {
        static_assert(kBins == 4 * kSelThreads, "four bins a thread");
        const int top = kBins - 1 - 4 * tid;  // this thread's bins: top, top - 1, top - 2, top - 3
        int32_t c4[4] = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < C; ++r) {
            const uint4 h = C > 1 ? peer_u128(&sm.hist[top - 3], r)
                                  : *reinterpret_cast<const uint4 *>(&sm.hist[top - 3]);
            c4[0] += (int32_t)h.w;
            c4[1] += (int32_t)h.z;
            c4[2] += (int32_t)h.y;
            c4[3] += (int32_t)h.x;
        }
        int32_t total;
        int32_t above = block_exclusive_scan<kSelThreads>((c4[0] + c4[1]) + (c4[2] + c4[3]), sm.scan, &total);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (above < K && K <= above + c4[e]) {
                sm.pick[0] = top - e;
                sm.pick[1] = above;
                sm.pick[2] = c4[e];
            }
            above += c4[e];
        }
        __syncthreads();
    }
    const uint32_t bin = sm.pick[0];
    int32_t left = K - (int32_t)sm.pick[1];  // to take of the bin's rows
    const int32_t n_bin = (int32_t)sm.pick[2];
    // the K-th largest key: rows with a larger one are taken, those with an
    // equal one in row order while `left` lasts
    uint32_t kth = 0u;
    // rows above the threshold and on it in the CTAs before this one
    uint32_t gt_before = 0, eq_before = 0;
    if (n_bin <= kCand) {
        uint32_t n_gt = 0;
        sweep([&](float s) {
            const uint32_t b = bin_of(s);
            n_gt += b > bin;
            if (b == bin) sm.cand[atomicAdd(&sm.n_cand, 1u)] = row_key(s);
        });
        n_gt = __reduce_add_sync(0xffffffffu, n_gt);
        if (C > 1 && lane == 0) atomicAdd(&sm.counts[0], n_gt);
        sync();
        const uint32_t m = gather(&sm.n_cand, 0u);  // lane r: CTA r's candidates
        if (warp < C) {  // warp w fetches CTA w's
            const uint32_t at = __reduce_add_sync(0xffffffffu, lane < warp ? m : 0u);
            const uint32_t mine = __shfl_sync(0xffffffffu, m, warp);
            for (uint32_t i = lane; i < mine; i += 32)
                sm.all[at + i] = C > 1 ? peer_u32(&sm.cand[i], warp) : sm.cand[i];
        }
        uint32_t start = 0;  // candidates of the CTAs before this one
        if (C > 1) {
            const uint32_t pg = gather(&sm.counts[0], 0u);
            gt_before = __reduce_add_sync(0xffffffffu, lane < rank ? pg : 0u);
            start = __reduce_add_sync(0xffffffffu, lane < rank ? m : 0u);
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // done with the peers
        }
        __syncthreads();
        if (tid < n_bin) {
            const uint32_t mine = sm.all[tid];
            int32_t gt = 0, eq = 0;
            for (int32_t i = 0; i < n_bin; ++i) {
                gt += sm.all[i] > mine;
                eq += sm.all[i] == mine;
            }
            if (gt < left && left <= gt + eq) {  // all that pass hold the same key
                sm.pick[0] = mine;
                sm.pick[1] = gt;
            }
        }
        __syncthreads();
        kth = sm.pick[0];
        left -= (int32_t)sm.pick[1];
        if (C > 1) {
            const bool in = (uint32_t)tid < start;
            const uint32_t k = in ? sm.all[tid] : 0u;
            gt_before += __syncthreads_count(in && k > kth);
            eq_before = __syncthreads_count(in && k == kth);
        }
    } else {
        uint32_t mask = 0u;  // bits of kth that are known
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            uint32_t *h = sm.digit[pass & 1];
            sweep([&](float s) {
                const uint32_t k = row_key(s);
                if (bin_of(s) == bin && (k & mask) == kth) atomicAdd(&h[(k >> shift) & 255u], 1u);
            });
            if (tid < 256) sm.digit[(pass + 1) & 1][tid] = 0;  // by all, in the pass before
            sync();
            int32_t cnt = 0;
            if (tid < 256)
#pragma unroll
                for (int r = 0; r < C; ++r)
                    cnt += (int32_t)(C > 1 ? peer_u32(&h[255 - tid], r) : h[255 - tid]);
            int32_t total;
            const int32_t above = block_exclusive_scan<kSelThreads>(cnt, sm.scan, &total);
            if (tid < 256 && above < left && left <= above + cnt) {
                sm.pick[0] = 255 - tid;
                sm.pick[1] = above;
            }
            sync();  // the peers have read this pass's counts
            kth |= sm.pick[0] << shift;
            mask |= 255u << shift;
            left -= (int32_t)sm.pick[1];
            __syncthreads();
        }
        if (C > 1) {
            uint32_t n_gt = 0, n_eq = 0;
            sweep([&](float s) {
                const uint32_t k = row_key(s);
                n_gt += k > kth;
                n_eq += k == kth;
            });
            n_gt = __reduce_add_sync(0xffffffffu, n_gt);
            n_eq = __reduce_add_sync(0xffffffffu, n_eq);
            if (lane == 0) {
                atomicAdd(&sm.counts[0], n_gt);
                atomicAdd(&sm.counts[1], n_eq);
            }
            sync();
            const uint32_t pg = gather(&sm.counts[0], 0u), pe = gather(&sm.counts[1], 0u);
            gt_before = __reduce_add_sync(0xffffffffu, lane < rank ? pg : 0u);
            eq_before = __reduce_add_sync(0xffffffffu, lane < rank ? pe : 0u);
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // done with the peers
        }
    }
    // ---- emission in row order
    for (int32_t c0 = r0; c0 < r1; c0 += kSelRows) {
        if (!kHeld) fetch(c0);
        uint32_t up = 0, on = 0;  // this thread's rows above the K-th key and on it
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            const int32_t r = row_at(c0, i);
            const float v[4] = {held[i].x, held[i].y, held[i].z, held[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t k = row_key(v[e]), bit = 1u << (4 * i + e);
                if (r + e < r1 && k > kth) up |= bit;
                if (r + e < r1 && k == kth) on |= bit;
            }
        }
        // packed counts: a chunk's rows stay below 2^16
        static_assert(kSelThreads / 32 <= 32 && kSelRows < 65536, "packed counts");
        const uint32_t mine = (uint32_t)__popc(up) | ((uint32_t)__popc(on) << 16);
        uint32_t x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) sm.warps[warp] = x;
        __syncthreads();
        const uint32_t others = lane < kSelThreads / 32 ? sm.warps[lane] : 0u;
        const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? others : 0u) + x - mine;
        const uint32_t chunk = __reduce_add_sync(0xffffffffu, others);
        uint32_t g1 = gt_before + (before & 0xffffu), e1 = eq_before + (before >> 16);
        gt_before += chunk & 0xffffu;
        eq_before += chunk >> 16;
        for (uint32_t todo = up | on; todo; todo &= todo - 1) {
            const int i = __ffs(todo) - 1;
            const bool above = (up >> i) & 1u;
            if (above || e1 < (uint32_t)left) {
                const uint32_t at = g1 + min(e1, (uint32_t)left);
                const int32_t r = row_at(c0, 0) + i;
                idx[at] = r;
                if (val) val[at] = sc[r];
            }
            g1 += above;
            e1 += !above;
        }
    }
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // peers are done with sm
}

template <int C>
cudaError_t launch_select(const IndexerPagedArgs &a, bool held, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.T * C);
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    return held ? cudaLaunchKernelEx(&cfg, indexer_paged_select_kernel<C, true>, a)
                : cudaLaunchKernelEx(&cfg, indexer_paged_select_kernel<C, false>, a);
}

template <int DI>
cudaError_t allow_smem() {
    return cudaFuncSetAttribute(indexer_paged_score_kernel<DI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)Score<DI>::kSmem);
}

}  // namespace

size_t indexer_paged_workspace_bytes(int32_t T, int64_t max_rows) {
    return (size_t)T * (size_t)((max_rows + 63) / 64 * 64) * sizeof(float);
}

cudaError_t launch_indexer_topk_paged(IndexerPagedArgs a, cudaStream_t stream) {
    a.row_pad = ((int64_t)a.max_rows + 63) / 64 * 64;
    static PerContext pc;
    int sms, dev;
    bool first;
    unsigned long long ctx;
    cudaError_t e = enter_context(pc, &first, &ctx, &dev);
    if (e == cudaSuccess) e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    if (first) {
        if ((e = allow_smem<64>()) != cudaSuccess || (e = allow_smem<128>()) != cudaSuccess) return e;
        entered_context(pc, dev, ctx);
    }
    const bool scored = a.max_rows > 0 && (a.max_rows > a.topk || a.topk_val);
    if (scored) {
        e = a.Di == 128 ? launch_early(indexer_paged_score_kernel<128>, dim3(sms), dim3(kThreads),
                                       Score<128>::kSmem, stream, a)
                        : launch_early(indexer_paged_score_kernel<64>, dim3(sms), dim3(kThreads),
                                       Score<64>::kSmem, stream, a);
        if (e != cudaSuccess) return e;
    }
    // CTAs a token: as few as hold the longest row the table allows in their
    // registers (a cluster's barriers and words cost more than its CTAs save:
    // whole calls of one token over 32768 rows 14.2 us, 16.0 with twice the
    // CTAs; of 64 tokens over up to 16384 rows 39.4 us, 41.0 with twice).
    int C = 1;
    while (C < kMaxCluster && (int64_t)C * kSelRows < a.max_rows) C *= 2;
    const bool held = (int64_t)C * kSelRows >= a.max_rows;
    switch (C) {
        case 1: return launch_select<1>(a, held, stream);
        case 2: return launch_select<2>(a, held, stream);
        case 4: return launch_select<4>(a, held, stream);
        default: return launch_select<8>(a, held, stream);
    }
}

}  // namespace csa
