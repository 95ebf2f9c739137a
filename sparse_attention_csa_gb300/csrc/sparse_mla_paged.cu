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
#include "tc_ptx.cuh"

namespace csa {

namespace {

constexpr int kTile = 64;
constexpr int kMaxGrid = 160;  // CTAs of the persistent grid (sizes the workspace)
constexpr int kThreads = 352;  // 8 softmax and epilogue warps, 2 loader warps, 1 MMA warp
constexpr int kLoaders = 64;
constexpr int kMmaWarp = 10;
constexpr int kPieces = 64;    // pieces of a run described in shared memory at a time
constexpr float kLazyMax = 8.0f;  // base-2 units
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// shared memory map (offsets from a 1024-byte aligned base)
constexpr uint32_t kOffQ = 0;            // 8 chunks x [64 heads x 128 B]
constexpr uint32_t kOffKV = 65536;       // 2 stages x 8 chunks x [64 rows x 128 B]
constexpr uint32_t kStage = 65536;
constexpr uint32_t kOffP = 196608;       // 2 x [64 rows x 64 heads] bf16, MN-major
constexpr uint32_t kOffMisc = 212992;

// tensor memory columns
constexpr uint32_t kColS = 0;            // 2 x 64
constexpr uint32_t kColO = 256;          // 4 slabs of 128 d x 64 heads
constexpr uint32_t kTmemCols = 512;

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

// A stretch of tiles [j0, j1) of one token, worked by one CTA.
struct Piece {
    int32_t t, j0, j1;
    int32_t slot;  // workspace slot, or -1: the whole token
    Keys k;
};

struct Misc {
    uint64_t q_full, q_empty;
    uint64_t kv_full[2], kv_empty[2];
    uint64_t s_full[2], p_full[2];
    uint64_t o_full, o_empty, drain;
    uint32_t tmem_base;
    int32_t abort;
    int64_t run_base;        // tiles before token run_t
    int32_t run_t;           // token holding the CTA's next tile
    int32_t scan[kThreads / 32 + 1];
    uint32_t valid[2][2];    // per stage and loader warp: 32 slot bits
    Piece piece[kPieces];
    int32_t n_pieces;
    alignas(16) float red[2][4][64];  // [tile parity][lane quarter][head]
    float sink2[64];                  // sink * log2(e), -inf when absent
};

constexpr size_t kSmemBytes = kOffMisc + sizeof(Misc) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct Ctx {
    Misc *m;
    int32_t *err;
    uint64_t limit;  // pipeline waits give up after this long
    __device__ __forceinline__ bool aborted() const {
        return *reinterpret_cast<volatile int32_t *>(&m->abort) != 0;
    }
    __device__ __forceinline__ void fail(int site) const {
        *reinterpret_cast<volatile int32_t *>(&m->abort) = 1;
        report_error(err, kErrTimeout, kKerMlaPaged, site);
    }
    // bounded wait; false (and abort) on timeout or when already aborted
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, int site) const {
        if (aborted()) return false;
        if (tc::mbar_wait(bar, parity, limit)) return true;
        fail(site);
        return false;
    }
};

// AND / OR of v over the 128 threads of named barrier `id`.
__device__ __forceinline__ bool bar_and(uint32_t id, bool v) {
    uint32_t out;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(out)
        : "r"((uint32_t)v), "r"(id)
        : "memory");
    return out != 0;
}
__device__ __forceinline__ bool bar_or(uint32_t id, bool v) { return !bar_and(id, !v); }

// The mbarrier counts one arrival (already included in its expected count)
// once every cp.async this thread issued so far has landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar))
                 : "memory");
}

// 32 values per thread -> lane L holds the warp-wide reduction of value L:
// each step sends the half of the values the partner keeps.
template <bool kMax>
__device__ __forceinline__ float reduce_scatter(const float (&x)[32], int lane) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = x[i];
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) {
        const bool hi = lane & w;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, hi ? v[i] : v[w + i], w);
            const float mine = hi ? v[w + i] : v[i];
            v[i] = kMax ? fmaxf(mine, other) : mine + other;
        }
    }
    return v[0];
}

__global__ void __launch_bounds__(kThreads, 1)
sparse_mla_paged_kernel(const __grid_constant__ MlaPagedArgs a) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc *ms = reinterpret_cast<Misc *>(smem + kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Space ws(a.workspace, a.H);
    const Ctx cx{ms, a.err, a.wait_ns};
    const int32_t c = blockIdx.x;

    if (tid == 0) {
        tc::mbar_init(&ms->q_full, kLoaders);
        tc::mbar_init(&ms->q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&ms->kv_full[i], kLoaders + 2);
            tc::mbar_init(&ms->kv_empty[i], 1);
            tc::mbar_init(&ms->s_full[i], 1);
            tc::mbar_init(&ms->p_full[i], 256);
        }
        tc::mbar_init(&ms->o_full, 1);
        tc::mbar_init(&ms->o_empty, 256);
        tc::mbar_init(&ms->drain, 1);
        ms->abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&ms->tmem_base, kTmemCols);
        tc::tmem_relinquish();
    }
    // heads past H: zero rows of Q, never written again
    for (int i = tid; i < (64 - a.H) * 64; i += kThreads) {
        const int h = a.H + (i >> 6), u = i & 63;
        *reinterpret_cast<uint4 *>(smem + kOffQ + (u >> 3) * 8192 + h * 128 + (u & 7) * 16) =
            make_uint4(0, 0, 0, 0);
    }
    // everything above is local: wait for the kernels before this one
    grid_dependency_wait();
    launch_dependents();
    if (tid < 64) ms->sink2[tid] = (a.sinks && tid < a.H) ? __ldg(a.sinks + tid) * kLog2e : -INFINITY;
    if (tid == 0) ws.join[c] = {-1, 0, 0, 0};
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = ms->tmem_base;

    // ------------------------------------------------ this CTA's run of tiles
    int64_t N = 0;
    for (int32_t t0 = 0; t0 < a.T; t0 += kThreads) {
        int32_t total;
        const int32_t t = t0 + tid;
        block_exclusive_scan<kThreads>(t < a.T ? token_keys(a, t, c == 0).tiles() : 0, ms->scan,
                                       &total);
        N += total;
    }
    const int64_t G = min((int64_t)gridDim.x, N);  // every run holds a tile
    const int64_t s = c < G ? c * N / G : N, e = c < G ? (c + 1) * N / G : N;
    if (s < e) {  // the token holding tile s
        int64_t base = 0;
        for (int32_t t0 = 0; t0 < a.T && base <= s; t0 += kThreads) {
            int32_t total;
            const int32_t t = t0 + tid, n = t < a.T ? token_keys(a, t, false).tiles() : 0;
            const int64_t b = base + block_exclusive_scan<kThreads>(n, ms->scan, &total);
            if (b <= s && s < b + n) {
                ms->run_t = t;
                ms->run_base = b;
            }
            base += total;
        }
    }
    __syncthreads();

    // counters of each role, kept across batches of pieces
    uint32_t g = 0, np = 0;
    bool issued = false;
    int64_t done = s;
    while (done < e) {
        // ------------------------------------------------- a batch of pieces
        const int32_t t_first = ms->run_t;
        const int64_t base = ms->run_base;
        {
            int32_t total;
            const int32_t t = t_first + tid;
            Keys k = {-1, 0, 0, 0, 0};
            int32_t n = 0;
            if (tid < kPieces && t < a.T) {
                k = token_keys(a, t, false);
                n = k.tiles();
            }
            const int64_t b = base + block_exclusive_scan<kThreads>(n, ms->scan, &total);
            if (n > 0 && b < e) {
                Piece p;
                p.t = t;
                p.j0 = (int32_t)max(s - b, (int64_t)0);
                p.j1 = (int32_t)min(e - b, (int64_t)n);
                p.slot = p.j0 == 0 && p.j1 == n ? -1 : 2 * c + (p.j0 == 0 ? 1 : 0);
                p.k = k;
                ms->piece[tid] = p;
                if (p.slot == 2 * c + 1)  // starts here, goes on in other CTAs
                    ws.join[c] = {t, c, (int32_t)(((b + n) * G - 1) / N), 0};
                if (tid == kPieces - 1 || t + 1 == a.T || b + n >= e) ms->n_pieces = tid + 1;
            }
            if (tid == 0) {
                ms->run_t = t_first + kPieces;
                ms->run_base = base + total;
            }
            done = min(e, base + total);
            __syncthreads();
        }
        const int32_t n_pieces = ms->n_pieces;

        if (warp == kMmaWarp) {
            // ===================================================== MMA warp
            if (lane == 0) {
                const uint32_t id_s = tc::idesc_bf16(64, 64, false, false);
                const uint32_t id_o = tc::idesc_bf16(128, 64, true, true);
                const uint64_t ds_a = tc::smem_desc(tc::smem_u32(smem + kOffKV), 16, 1024);
                const uint64_t ds_b = tc::smem_desc(tc::smem_u32(smem + kOffQ), 16, 1024);
                const uint64_t do_a = tc::smem_desc(tc::smem_u32(smem + kOffKV), 8192, 1024);
                const uint64_t do_b = tc::smem_desc(tc::smem_u32(smem + kOffP), 8192, 1024);
                // S^T of tile x, all 32 MMAs back to back
                auto scores = [&](uint32_t x, bool last) -> bool {
                    if (!cx.wait(&ms->kv_full[x & 1], (x >> 1) & 1, 21)) return false;
                    tc::fence_proxy_async_smem();  // cp.async wrote through the generic proxy
                    tc::tc_fence_after();
                    const uint32_t st = (x & 1) * kStage;
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc::mma_bf16(tmem + kColS + 64 * (x & 1),
                                         tc::desc_add(ds_a, st + ch * 8192 + kk * 32),
                                         tc::desc_add(ds_b, ch * 8192 + kk * 32), id_s, (ch | kk) != 0);
                    issued = true;
                    tc::mma_commit(&ms->s_full[x & 1]);
                    if (last) tc::mma_commit(&ms->q_empty);
                    return true;
                };
                bool ok = true;
                for (int32_t i = 0; i < n_pieces && ok; ++i, ++np) {
                    const int32_t n = ms->piece[i].j1 - ms->piece[i].j0;
                    ok = cx.wait(&ms->q_full, np & 1, 20) && scores(g, n == 1);
                    for (int32_t j = 0; j < n && ok; ++j, ++g) {
                        // the next tile's scores run while this one's softmax does
                        if (j + 1 < n && !(ok = scores(g + 1, j + 2 == n))) break;
                        ok = cx.wait(&ms->p_full[g & 1], (g >> 1) & 1, 22) &&
                             (j > 0 || cx.wait(&ms->o_empty, (np & 1) ^ 1, 23));
                        if (!ok) break;
                        tc::tc_fence_after();
                        const uint32_t st = (g & 1) * kStage, pb = (g & 1) * 8192;
#pragma unroll
                        for (int sl = 0; sl < 4; ++sl)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc::mma_bf16(tmem + kColO + 64 * sl,
                                             tc::desc_add(do_a, st + sl * 16384 + kk * 2048),
                                             tc::desc_add(do_b, pb + kk * 2048), id_o, (j | kk) != 0);
                        tc::mma_commit(&ms->kv_empty[g & 1]);
                    }
                    if (ok) tc::mma_commit(&ms->o_full);
                }
            }
            __syncwarp();
        } else if (warp >= 8) {
            // ================================================= loader warps
            // Warp w holds slots 32 w .. 32 w + 31 of every tile, looked up one
            // per lane, the next tile's while this one waits for its stage.
            const int w = warp - 8, li = tid - 256;
            bool ok = true;
            for (int32_t i = 0; i < n_pieces && ok; ++i, ++np) {
                const int32_t t = ms->piece[i].t, j0 = ms->piece[i].j0, j1 = ms->piece[i].j1;
                const Keys k = ms->piece[i].k;
                auto lookup = [&](int32_t j) {
                    return j < j1 ? key_row(a, k, t, j * kTile + 32 * w + lane) : nullptr;
                };
                const __nv_bfloat16 *rows = lookup(j0), *next = lookup(j0 + 1);
                ok = __all_sync(0xffffffffu, cx.wait(&ms->q_empty, (np & 1) ^ 1, 40));
                if (!ok) break;
                const __nv_bfloat16 *q = a.q + (int64_t)t * a.H * 512;
                for (int u = li; u < a.H * 64; u += kLoaders) {
                    const int h = u >> 6, ch = (u >> 3) & 7, x = u & 7;
                    tc::cp_async16_zfill(smem + kOffQ + ch * 8192 + h * 128 + ((x ^ (h & 7)) << 4),
                                         q + (int64_t)u * 8, 16);
                }
                cp_async_arrive(&ms->q_full);
                for (int32_t j = j0; j < j1; ++j, ++g) {
                    ok = __all_sync(0xffffffffu, cx.wait(&ms->kv_empty[g & 1], ((g >> 1) & 1) ^ 1, 41));
                    if (!ok) break;
                    const uint32_t m = __ballot_sync(0xffffffffu, rows != nullptr);
                    unsigned char *dst =
                        smem + kOffKV + (g & 1) * kStage + (lane >> 3) * 8192 + 32 * w * 128;
#pragma unroll 16
                    for (int r = 0; r < 32; ++r) {
                        const __nv_bfloat16 *src = reinterpret_cast<const __nv_bfloat16 *>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(rows), r));
                        const uint32_t bytes = src ? 16u : 0u;  // no key: zeros
                        if (!src) src = a.q;
                        unsigned char *d = dst + r * 128 + (((lane & 7) ^ (r & 7)) << 4);
                        tc::cp_async16_zfill(d, src + lane * 8, bytes);
                        tc::cp_async16_zfill(d + 4 * 8192, src + 256 + lane * 8, bytes);
                    }
                    cp_async_arrive(&ms->kv_full[g & 1]);
                    if (lane == 0) {
                        ms->valid[g & 1][w] = m;
                        tc::mbar_arrive(&ms->kv_full[g & 1]);
                    }
                    rows = next;
                    next = lookup(j + 2);
                }
            }
        } else {
            // =========================================== softmax + epilogue
            // Warpgroup wg: heads 32 wg .. 32 wg + 31. Lane quarter q4 of S^T
            // holds key slots 16 q4 .. 16 q4 + 15 in its first 16 lanes.
            const int wg = warp >> 2, q4 = warp & 3, h0 = 32 * wg;
            const uint32_t bar = 1 + wg;
            const uint32_t lane_addr = tmem + ((uint32_t)(32 * q4) << 16);
            const float sc = a.softmax_scale * kLog2e;
            bool ok = true, stop = false;
            for (int32_t i = 0; i < n_pieces && !stop; ++i, ++np) {
                const int32_t t = ms->piece[i].t, n = ms->piece[i].j1 - ms->piece[i].j0;
                const int32_t slot = ms->piece[i].slot;
                // m_lane: running maximum (base 2) of head h0 + lane; m_cur:
                // every thread's copy of all 32
                float m_lane = -INFINITY, lp[32], m_cur[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    lp[x] = 0.0f;
                    m_cur[x] = -INFINITY;
                }
                for (int32_t j = 0; j < n; ++j, ++g) {
                    ok = cx.wait(&ms->kv_full[g & 1], (g >> 1) & 1, 30) &&
                         cx.wait(&ms->s_full[g & 1], (g >> 1) & 1, 31);
                    tc::tc_fence_after();
                    const bool key =
                        lane < 16 && ((ms->valid[g & 1][q4 >> 1] >> (16 * (q4 & 1) + lane)) & 1u);
                    float v[32];
                    const uint32_t s_addr = lane_addr + kColS + 64 * (g & 1) + h0;
                    tc::tmem_ld32(s_addr, v);
                    tc::tmem_wait_ld();
                    // Scores in base 2 above the running maximum. The maximum
                    // moves only when a score exceeds it by more than kLazyMax
                    // (always at a token's first keys, where it is -inf), so
                    // that O^T is rarely rescaled; the warpgroup agrees on it.
                    bool over = !ok;
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        v[x] = key ? fmaf(v[x], sc, -m_cur[x]) : -INFINITY;
                        over |= v[x] > kLazyMax;
                    }
                    if (bar_or(bar, over)) {
                        if (j > 0) ok = ok && cx.wait(&ms->kv_empty[(g - 1) & 1], ((g - 1) >> 1) & 1, 33);
                        if (!bar_and(bar, ok)) {
                            stop = true;
                            break;
                        }
                        tc::tc_fence_after();
                        tc::tmem_ld32(s_addr, v);  // the scores again
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x) v[x] = key ? v[x] * sc : -INFINITY;
                        const uint32_t rs = g & 1;
                        ms->red[rs][q4][h0 + lane] = reduce_scatter<true>(v, lane);
                        tc::named_bar_sync(bar, 128);
                        const float mt = fmaxf(fmaxf(ms->red[rs][0][h0 + lane], ms->red[rs][1][h0 + lane]),
                                               fmaxf(ms->red[rs][2][h0 + lane], ms->red[rs][3][h0 + lane]));
                        // the first keys set the maximum itself: the largest
                        // weight is then exactly 1 in bf16
                        const bool up = mt > m_lane + kLazyMax;
                        const float al_lane = up && m_lane != -INFINITY ? tc::ex2_approx(m_lane - mt) : 1.0f;
                        const bool scale = __any_sync(0xffffffffu, up && m_lane != -INFINITY);
                        if (up) m_lane = mt;
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            m_cur[x] = __shfl_sync(0xffffffffu, m_lane, x);
                            lp[x] *= __shfl_sync(0xffffffffu, al_lane, x);
                            v[x] = m_cur[x] == -INFINITY ? -INFINITY : v[x] - m_cur[x];
                        }
                        if (scale) {
#pragma unroll 1
                            for (int sl = 0; sl < 4; ++sl) {
                                float o[32];
                                const uint32_t addr = lane_addr + kColO + 64 * sl + h0;
                                tc::tmem_ld32(addr, o);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int x = 0; x < 32; ++x)
                                    o[x] *= __shfl_sync(0xffffffffu, al_lane, x);
                                tc::tmem_st32(addr, o);
                            }
                            tc::tmem_wait_st();
                        }
                    }
                    // weights (bf16) -> row of P^T: 64 bytes of its 128
                    const int row = 16 * q4 + (lane & 15);
                    unsigned char *prow = smem + kOffP + (g & 1) * 8192 + row * 128;
#pragma unroll
                    for (int cq = 0; cq < 4; ++cq) {
                        uint32_t w4[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int x = 8 * cq + 2 * y;
                            const float p0 = tc::ex2_approx(v[x]), p1 = tc::ex2_approx(v[x + 1]);
                            lp[x] += p0;
                            lp[x + 1] += p1;
                            const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
                            w4[y] = *reinterpret_cast<const uint32_t *>(&pb);
                        }
                        if (lane < 16)
                            *reinterpret_cast<uint4 *>(prow + (((4 * wg + cq) ^ (row & 7)) << 4)) =
                                make_uint4(w4[0], w4[1], w4[2], w4[3]);
                    }
                    tc::fence_proxy_async_smem();
                    tc::tc_fence_before();
                    tc::mbar_arrive(&ms->p_full[g & 1]);
                }
                if (stop) break;
                // ---- row sums, then O^T
                const uint32_t rs = g & 1;  // no softmax step of this token reads it any more
                ms->red[rs][q4][h0 + lane] = reduce_scatter<false>(lp, lane);
                tc::named_bar_sync(bar, 128);
                const float l_lane = (ms->red[rs][0][h0 + lane] + ms->red[rs][1][h0 + lane]) +
                                     (ms->red[rs][2][h0 + lane] + ms->red[rs][3][h0 + lane]);
                const bool mine = q4 == 0 && h0 + lane < a.H;
                float f_lane = 1.0f;  // O^T times this
                if (slot < 0) {
                    const float sk = ms->piece[i].k.seq >= 0 ? ms->sink2[h0 + lane] : -INFINITY;
                    const float M = fmaxf(m_lane, sk);
                    const float f = m_lane == -INFINITY ? 0.0f : tc::ex2_approx(m_lane - M);
                    const float Z = fmaf(l_lane, f, sk == -INFINITY ? 0.0f : tc::ex2_approx(sk - M));
                    f_lane = Z > 0.0f ? f / Z : 0.0f;
                    if (mine && a.lse) a.lse[(int64_t)t * a.H + h0 + lane] = (M + tc::lg2_approx(Z)) * kLn2;
                } else if (mine) {
                    ws.m[slot * a.H + h0 + lane] = m_lane;
                    ws.l[slot * a.H + h0 + lane] = l_lane;
                }
                float fac[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) fac[x] = __shfl_sync(0xffffffffu, f_lane, x);
                ok = cx.wait(&ms->o_full, np & 1, 32);
                if (!bar_and(bar, ok)) {
                    stop = true;
                    break;
                }
                tc::tc_fence_after();
                // Lane of O^T slab sl: d = 128 sl + 32 q4 + lane, 32 heads a thread
                const int n_h = min(32, a.H - h0), d = 32 * q4 + lane;
                __nv_bfloat16 *outp = a.out + ((int64_t)t * a.H + h0) * 512 + d;
                float *wsp = ws.o + ((int64_t)max(slot, 0) * a.H + h0) * 512 + d;
#pragma unroll 1
                for (int sl = 0; sl < 4; ++sl) {
                    float o[32];
                    tc::tmem_ld32(lane_addr + kColO + 64 * sl + h0, o);
                    tc::tmem_wait_ld();
                    if (sl == 3) {  // O^T is read: the next token's may start
                        tc::tc_fence_before();
                        tc::mbar_arrive(&ms->o_empty);
                    }
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        if (x >= n_h) break;
                        if (slot < 0)
                            outp[x * 512 + 128 * sl] = __float2bfloat16_rn(o[x] * fac[x]);
                        else
                            wsp[x * 512 + 128 * sl] = o[x];
                    }
                }
            }
        }
        __syncthreads();
        if (cx.aborted()) break;
    }

    // ------------------------------------------------------------- teardown
    if (warp == 8 || warp == 9) asm volatile("cp.async.wait_all;" ::: "memory");
    if (tid == 32 * kMmaWarp && issued) {  // every MMA issued is done before tensor memory is freed
        tc::mma_commit(&ms->drain);
        if (!tc::mbar_wait(&ms->drain, 0)) cx.fail(24);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

// Block (c, y): heads 8y .. 8y + 7 of the token whose first tile CTA c held
// and that other CTAs went on with; one warp per head, 16 dims per lane.
__global__ void __launch_bounds__(256) sparse_mla_paged_join_kernel(MlaPagedArgs a) {
    const Space ws(a.workspace, a.H);
    grid_dependency_wait();
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
    e = cudaFuncSetAttribute(sparse_mla_paged_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    const int grid = min(sms, kMaxGrid);
    e = launch_early(sparse_mla_paged_kernel, dim3(grid), dim3(kThreads), kSmemBytes, stream, a);
    if (e != cudaSuccess) return e;
    return launch_early(sparse_mla_paged_join_kernel, dim3(grid, (a.H + 7) / 8), dim3(256), 0, stream, a);
}

}  // namespace csa
