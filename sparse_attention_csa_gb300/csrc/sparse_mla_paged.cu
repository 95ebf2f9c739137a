// Sparse MLA attention of new tokens over paged caches (sm_103a, tcgen05
// tensor cores, cp.async gathers): the keys of token t are the window rows of
// its sequence in the original-KV cache and the listed (or every visible) rows
// of the compressed cache.
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
//
// A tile. All heads share a row, which is both key and value, so the products
// are transposed, with the tile on the MMA's M side, and a tile is loaded once
// for both:
//     S^T: keys x heads, K = 512.  64 keys fill half of M = 128, which costs
//          the tensor core as much as all of it, so the other half of M takes
//          the same keys' dims 256-511 and N = 128 the heads against the low
//          and the high dims of Q: 16 MMAs (64 cycles each) in place of 32 (58
//          each). Of the four blocks of the result the two matching ones are
//          added. Rows of the low and the high half alternate in groups of 8,
//          so a key's two partial scores sit 8 lanes apart in one warp.
//     O^T: 4 slabs of 128 dims x 64 heads, K = 64 keys, the same bytes read
//          MN-major.
// Shared memory holds Q (64 KB), two tiles (128 KB) and two P (16 KB); tensor
// memory two S^T (256 columns) and O^T (256). The scores of a tile are issued
// while the previous tile's softmax runs. Rows are gathered by cp.async; their
// pages are found some tiles ahead by a warp of its own.
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "tc_ptx.cuh"
#include "tmap.h"

namespace csa {

namespace {

constexpr int kTile = 64;
constexpr int kMaxGrid = 160;     // CTAs of the persistent grid (sizes the workspace)
constexpr int kThreads = 384;     // 8 softmax and epilogue warps, 2 loaders, 1 MMA, 1 look-up
constexpr int kLoaders = 64;
constexpr int kMmaWarp = 10;
constexpr int kFindWarp = 11;
constexpr int kRing = 4;          // tiles whose rows are found ahead of the loaders
constexpr int kPieces = 64;       // pieces of a run described in shared memory at a time
constexpr float kLazyMax = 8.0f;  // base-2 units
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// shared memory map (offsets from a 1024-byte aligned base)
constexpr uint32_t kOffQ = 0;       // 4 dim groups x [low, high] x [64 heads x 128 B]
constexpr uint32_t kOffKV = 65536;  // 2 stages x 4 dim groups x 8 x [low, high] x [8 keys x 128 B]
constexpr uint32_t kStage = 65536;
constexpr uint32_t kOffP = 196608;  // 2 x [64 keys x 64 heads] bf16, MN-major
constexpr uint32_t kOffMisc = 212992;

// tensor memory columns
constexpr uint32_t kColS = 0;    // 2 x 128
constexpr uint32_t kColO = 256;  // 4 slabs of 128 d x 64 heads
constexpr uint32_t kTmemCols = 512;

struct Join {
    int32_t t, first, last, pad;  // token split over CTAs first..last (t < 0: none)
};

// Workspace: Join [kMaxGrid], then m and l [2 kMaxGrid][64], then the sums
// [2 kMaxGrid][ceil(H / 4)][512][4 heads]: a thread of the epilogue holds one
// dim of 32 heads, so a warp writes 512 bytes at once.
struct Space {
    Join *join;
    float *m, *l, *o;
    int32_t quads;
    __host__ __device__ Space(void *p, int32_t H) {
        join = static_cast<Join *>(p);
        m = reinterpret_cast<float *>(join + kMaxGrid);
        l = m + 2 * kMaxGrid * 64;
        o = l + 2 * kMaxGrid * 64;
        quads = (H + 3) / 4;
    }
    // four heads of one dim
    __device__ __forceinline__ float4 *sums(int32_t slot, int32_t quad, int32_t d) const {
        return reinterpret_cast<float4 *>(o) + ((int64_t)slot * quads + quad) * 512 + d;
    }
};

// Key slots of a token, from its position alone.
struct Keys {
    int32_t seq, win_start, n_win, vis, n_cmp;
    __device__ __forceinline__ uint32_t slots() const { return (uint32_t)n_win + (uint32_t)n_cmp; }
    __device__ __forceinline__ int32_t tiles() const {  // a token without keys has one, empty
        return max(1, (int32_t)(((uint32_t)n_win + (uint32_t)n_cmp + kTile - 1) / kTile));
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
        const int32_t cap = a.cmp.max_pages * a.cmp.page_size;
        k.vis = (int32_t)(((uint32_t)pos + 1u) / (uint32_t)a.cmp_ratio);
        if (k.vis > cap) {
            if (report) report_error(a.err, kErrCheck, kKerMlaPaged, 2);
            k.vis = cap;
        }
        k.n_cmp = a.idx ? (k.vis > 0 ? a.topk : 0) : k.vis;
    }
    return k;
}

// Finding the pool row of a key slot takes two dependent loads (the list's
// entry, the page). They are three steps, so that those of later tiles stay in
// flight: slot_row -> slot_page -> slot_ptr.
struct Slot {
    int32_t in;    // row within its page; -1: no key
    int32_t phys;  // page of the pool
    bool win;      // of the original-KV cache
};

// Row of the sequence in key slot i, -1 past the last slot; a list's entry is
// not checked yet.
__device__ __forceinline__ int32_t slot_row(const MlaPagedArgs &a, const Keys &k, int32_t t, uint32_t i) {
    if (i < (uint32_t)k.n_win) return k.win_start + (int32_t)i;
    if (i >= k.slots()) return -1;
    const int32_t e = (int32_t)(i - (uint32_t)k.n_win);
    return a.idx ? __ldg(a.idx + (int64_t)t * a.topk + e) : e;
}

__device__ __forceinline__ Slot slot_page(const MlaPagedArgs &a, const Keys &k, uint32_t i, int32_t row) {
    const bool win = i < (uint32_t)k.n_win;
    if (row < 0 || (!win && row >= k.vis)) return {-1, -1, win};
    const PagedRows &p = win ? a.ori : a.cmp;
    const uint32_t pg = (uint32_t)row / (uint32_t)p.page_size;
    const int32_t in = row - (int32_t)pg * p.page_size;
    return {in, pg < (uint32_t)p.max_pages ? __ldg(p.pages + (int64_t)k.seq * p.max_pages + pg) : -1, win};
}

// nullptr: no key, or its page is absent (recorded)
__device__ __forceinline__ const __nv_bfloat16 *slot_ptr(const MlaPagedArgs &a, const Slot &s) {
    if (s.in < 0) return nullptr;
    const PagedRows &p = s.win ? a.ori : a.cmp;
    if ((uint32_t)s.phys >= (uint32_t)p.num_pages) {
        report_error(a.err, kErrCheck, kKerMlaPaged, 3);
        return nullptr;
    }
    return p.base + ((int64_t)s.phys * p.page_size + s.in) * 512;
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
    uint64_t ring_full[kRing], ring_empty[kRing];
    const __nv_bfloat16 *ring[kRing][kTile];  // pool rows of a tile's slots, nullptr: no key
    uint32_t tmem_base;
    int32_t abort;
    int64_t run_base;      // tiles before token run_t
    int64_t done;          // tiles up to the end of the batch
    int32_t run_t;         // token holding the CTA's next tile
    int32_t n_pieces;
    int32_t scan[kThreads / 32 + 1];
    uint32_t valid[2][2];  // per stage and loader warp: 32 slot bits
    Piece piece[kPieces];
    alignas(16) float red[2][4][64];  // [tile parity][lane quarter][head]
    alignas(16) float m[64];          // running maximum (base 2)
    alignas(16) float fac[64];        // a rescaling's or the epilogue's factor
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

// 16 bytes global -> shared; `bytes` 0 writes zeros (nothing is read then).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// The mbarrier counts one arrival (already included in its expected count)
// once every cp.async this thread issued so far has landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar))
                 : "memory");
}

// Heads of one thread: 16 of its warpgroup's 32, by bit 3 of its lane. The 16
// lanes that agree in that bit hold 16 keys of the same heads:
// reduces each of the 16 values over them; a lane keeps value sum_index(lane).
template <bool kMax>
__device__ __forceinline__ float reduce_scatter16(const float (&x)[16], int lane) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = x[i];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int bit = s == 0 ? 16 : 8 >> s, w = 8 >> s;  // bits 4, 2, 1, 0; 8, 4, 2, 1 values kept
        const bool hi = lane & bit;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, hi ? v[i] : v[w + i], bit);
            const float mine = hi ? v[w + i] : v[i];
            v[i] = kMax ? fmaxf(mine, other) : mine + other;
        }
    }
    return v[0];
}
__device__ __forceinline__ int sum_index(int lane) { return ((lane >> 4) << 3) | (lane & 7); }

__global__ void __launch_bounds__(kThreads, 1)
sparse_mla_paged_kernel(const __grid_constant__ CUtensorMap q_map,
                        const __grid_constant__ MlaPagedArgs a) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc *ms = reinterpret_cast<Misc *>(smem + kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Space ws(a.workspace, a.H);
    const Ctx cx{ms, a.err, a.wait_ns};
    const int32_t c = blockIdx.x;

    if (tid == 0) {
        tc::mbar_init(&ms->q_full, 1);
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
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(&ms->ring_full[i], 32);
            tc::mbar_init(&ms->ring_empty[i], kLoaders);
        }
        ms->abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&ms->tmem_base, kTmemCols);
        tc::tmem_relinquish();
        if (lane == 0) tc::tma_prefetch_desc(&q_map);
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
    if (tid == 0) ws.join[c] = {-1, 0, 0, 0};
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();

    // ------------------------------------------------ this CTA's run of tiles
    // Tokens are scanned kThreads at a time; with no more than that, one scan
    // both counts the tiles and places them.
    const bool one_scan = a.T <= kThreads;
    Keys k = {-1, 0, 0, 0, 0};
    int32_t n = 0, total = 0;
    int64_t N = 0, b = 0;
    for (int32_t t0 = 0; t0 < a.T; t0 += kThreads) {
        const int32_t t = t0 + tid;
        n = 0;
        if (t < a.T) {
            k = token_keys(a, t, c == 0);
            n = k.tiles();
        }
        b = block_exclusive_scan<kThreads>(n, ms->scan, &total);
        N += total;
    }
    tc::tc_fence_after();
    const uint32_t tmem = ms->tmem_base;
    const int64_t per = div64(N + gridDim.x - 1, gridDim.x);  // tiles of a run
    const int64_t s = min(c * per, N), e = min(s + per, N);
    if (s == e) {  // no run left for this CTA
        __syncthreads();
        if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
        return;
    }
    if (one_scan) {
        if (b <= s && s < b + n) ms->run_t = tid;
    } else {  // the token holding tile s
        int64_t base = 0;
        for (int32_t t0 = 0; t0 < a.T && base <= s; t0 += kThreads) {
            const int32_t t = t0 + tid, nt = t < a.T ? token_keys(a, t, false).tiles() : 0;
            const int64_t bt = base + block_exclusive_scan<kThreads>(nt, ms->scan, &total);
            if (bt <= s && s < bt + nt) {
                ms->run_t = t;
                ms->run_base = bt;
            }
            base += total;
        }
    }
    __syncthreads();

    // counters of each role, kept across batches of pieces
    uint32_t g = 0, np = 0, nq = 0;
    bool issued = false;
    int64_t done = s;
    while (done < e) {
        // ------------------------------------------------- a batch of pieces
        const int32_t t_first = ms->run_t;
        int32_t t = tid;
        int x = tid - t_first;  // place in the batch
        if (!one_scan) {
            const int64_t base = ms->run_base;
            t = t_first + tid;
            x = tid;
            n = 0;
            if (tid < kPieces && t < a.T) {
                k = token_keys(a, t, false);
                n = k.tiles();
            }
            b = base + block_exclusive_scan<kThreads>(n, ms->scan, &total);
        }
        if (x >= 0 && x < kPieces && n > 0 && b < e) {
            Piece p;
            p.t = t;
            p.j0 = (int32_t)max(s - b, (int64_t)0);
            p.j1 = (int32_t)min(e - b, (int64_t)n);
            p.slot = p.j0 == 0 && p.j1 == n ? -1 : 2 * c + (p.j0 == 0 ? 1 : 0);
            p.k = k;
            ms->piece[x] = p;
            if (p.slot == 2 * c + 1)  // starts here, goes on in other CTAs
                ws.join[c] = {t, c, (int32_t)div64(b + n - 1, per), 0};
            if (x == kPieces - 1 || t + 1 == a.T || b + n >= e) {
                ms->n_pieces = x + 1;
                ms->done = min(e, b + n);
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
            // ================================================ Q and MMA warp
            if (lane == 0) {
                constexpr uint32_t id_s = tc::idesc_bf16(128, 128, false, false);
                constexpr uint32_t id_o = tc::idesc_bf16(128, 64, true, true);
                const uint64_t ds_a = tc::smem_desc(tc::smem_u32(smem + kOffKV), 16, 1024);
                const uint64_t ds_b = tc::smem_desc(tc::smem_u32(smem + kOffQ), 16, 1024);
                const uint64_t do_a = tc::smem_desc(tc::smem_u32(smem + kOffKV), 1024, 2048);
                const uint64_t do_b = tc::smem_desc(tc::smem_u32(smem + kOffP), 8192, 1024);
                auto load_q = [&](int32_t i) {  // rows past H stay zero
                    ++nq;
                    tc::mbar_expect_tx(&ms->q_full, (uint32_t)a.H * 1024u);
                    for (int ch = 0; ch < 8; ++ch)
                        tc::tma_load_3d(smem + kOffQ + (ch & 3) * 16384 + (ch >> 2) * 8192, &q_map,
                                        &ms->q_full, 64 * ch, 0, ms->piece[i].t);
                };
                bool ok = true;
                if (np == 0) load_q(0);
                for (int32_t i = 0; i < n_pieces && ok; ++i, ++np) {
                    const int32_t nt = ms->piece[i].j1 - ms->piece[i].j0;
                    if (i == 0 && np > 0) {  // a later batch's first piece
                        if (!(ok = cx.wait(&ms->q_empty, (np & 1) ^ 1, 25))) break;
                        load_q(0);
                    }
                    if (!(ok = cx.wait(&ms->q_full, np & 1, 20))) break;
                    // O^T of tile jo and scores of tile js, whichever is ready
                    // first, O^T before scores: it frees a stage, and the load
                    // that follows is the longest part of a tile's way.
                    int32_t js = 0, jo = 0;
                    const uint32_t g0 = g;
                    uint64_t since = 0;
                    while (jo < nt) {
                        const uint32_t xs = g0 + js, xo = g0 + jo;
                        if (jo < js && tc::mbar_try_wait(&ms->p_full[xo & 1], (xo >> 1) & 1, 20)) {
                            if (jo == 0 && !(ok = cx.wait(&ms->o_empty, (np & 1) ^ 1, 23))) break;
                            tc::tc_fence_after();
                            const uint32_t st = (xo & 1) * kStage, pb = (xo & 1) * 8192;
#pragma unroll
                            for (int d = 0; d < 4; ++d) {
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    tc::mma_bf16(tmem + kColO + 64 * d,
                                                 tc::desc_add(do_a, st + d * 16384 + kk * 4096),
                                                 tc::desc_add(do_b, pb + kk * 2048), id_o, (jo | kk) != 0);
                            }
                            tc::mma_commit(&ms->kv_empty[xo & 1]);
                            ++jo;
                            since = 0;
                            continue;
                        }
                        if (js < nt && js <= jo + 1 &&
                            tc::mbar_try_wait(&ms->kv_full[xs & 1], (xs >> 1) & 1, 20)) {
                            tc::fence_proxy_async_smem();  // cp.async wrote through the generic proxy
                            tc::tc_fence_after();
                            const uint32_t st = (xs & 1) * kStage;
#pragma unroll
                            for (int d = 0; d < 4; ++d)
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    tc::mma_bf16(tmem + kColS + 128 * (xs & 1),
                                                 tc::desc_add(ds_a, st + d * 16384 + kk * 32),
                                                 tc::desc_add(ds_b, d * 16384 + kk * 32), id_s,
                                                 (d | kk) != 0);
                            issued = true;
                            tc::mma_commit(&ms->s_full[xs & 1]);
                            since = 0;
                            if (++js == nt) {  // Q is read: the next piece's, under this O^T
                                tc::mma_commit(&ms->q_empty);
                                if (i + 1 < n_pieces) {
                                    if (!(ok = cx.wait(&ms->q_empty, np & 1, 25))) break;
                                    load_q(i + 1);
                                }
                            }
                            continue;
                        }
                        const uint64_t now = tc::globaltimer();
                        if (since == 0) since = now;
                        if (cx.aborted() || now - since > cx.limit) {
                            if (!cx.aborted()) cx.fail(21);
                            ok = false;
                            break;
                        }
                    }
                    if (!ok) break;
                    g = g0 + nt;
                    tc::mma_commit(&ms->o_full);
                }
            }
            __syncwarp();
        } else if (warp == 8 || warp == 9) {
            // ================================================= loader warps
            // Warp w copies slots 32 w .. 32 w + 31 of every tile.
            const int w = warp - 8;
            bool ok = true;
            for (int32_t i = 0; i < n_pieces && ok; ++i) {
                const int32_t nt = ms->piece[i].j1 - ms->piece[i].j0;
                for (int32_t j = 0; j < nt; ++j, ++g) {
                    ok = __all_sync(0xffffffffu,
                                    cx.wait(&ms->ring_full[g % kRing], (g / kRing) & 1, 40));
                    if (!ok) break;
                    const __nv_bfloat16 *mine = ms->ring[g % kRing][32 * w + lane];
                    tc::mbar_arrive(&ms->ring_empty[g % kRing]);
                    const uint32_t m = __ballot_sync(0xffffffffu, mine != nullptr);
                    ok = __all_sync(0xffffffffu, cx.wait(&ms->kv_empty[g & 1], ((g >> 1) & 1) ^ 1, 41));
                    if (!ok) break;
                    // Half a row (512 bytes) an instruction: pieces of 128 bytes
                    // of several rows took twice as long to issue. Lane: dim
                    // group lane / 8, 16-byte unit lane % 8 of its 128 bytes.
                    const uint32_t stage = tc::smem_u32(smem + kOffKV + (g & 1) * kStage) +
                                           (lane >> 3) * 16384 + w * 4 * 2048;
                    const int u = lane & 7;
#pragma unroll
                    for (int r = 0; r < 32; ++r) {
                        const __nv_bfloat16 *src = reinterpret_cast<const __nv_bfloat16 *>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), r));
                        const uint32_t bytes = src ? 16u : 0u;  // no key: zeros
                        if (!src) src = a.q;
                        const uint32_t dst = stage + (r >> 3) * 2048 + (r & 7) * 128 + ((u ^ (r & 7)) << 4);
                        cp_async16(dst, src + lane * 8, bytes);
                        cp_async16(dst + 1024, src + 256 + lane * 8, bytes);
                    }
                    cp_async_arrive(&ms->kv_full[g & 1]);
                    if (lane == 0) {
                        ms->valid[g & 1][w] = m;
                        tc::mbar_arrive(&ms->kv_full[g & 1]);
                    }
                }
            }
        } else if (warp == kFindWarp) {
            // ================================================= look-up warp
            // Two slots a lane. While a tile's rows are handed to the loaders,
            // the pages of the next tile and the list entries of the one after
            // it are being read. (Sending for the rows themselves ahead of
            // their copies, by L2 prefetches, made long rows 2 to 5 % slower.)
            bool ok = true;
            for (int32_t i = 0; i < n_pieces && ok; ++i) {
                const int32_t tt = ms->piece[i].t, j0 = ms->piece[i].j0, j1 = ms->piece[i].j1;
                const Keys kt = ms->piece[i].k;
                auto at = [&](int32_t j, int x) { return (uint32_t)j * kTile + 32 * x + lane; };
                auto row_of = [&](int32_t j, int x) { return j < j1 ? slot_row(a, kt, tt, at(j, x)) : -1; };
                int32_t r0[2], r1[2], r2[2];
                Slot s0[2], s1[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    r0[x] = row_of(j0, x);
                    r1[x] = row_of(j0 + 1, x);
                    r2[x] = row_of(j0 + 2, x);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    s0[x] = slot_page(a, kt, at(j0, x), r0[x]);
                    s1[x] = slot_page(a, kt, at(j0 + 1, x), r1[x]);
                }
                for (int32_t j = j0; j < j1; ++j, ++g) {
                    ok = __all_sync(0xffffffffu,
                                    cx.wait(&ms->ring_empty[g % kRing], ((g / kRing) & 1) ^ 1, 50));
                    if (!ok) break;
                    const __nv_bfloat16 *row[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        row[x] = slot_ptr(a, s0[x]);
                        ms->ring[g % kRing][32 * x + lane] = row[x];
                    }
                    tc::mbar_arrive(&ms->ring_full[g % kRing]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        s0[x] = s1[x];
                        s1[x] = slot_page(a, kt, at(j + 2, x), r2[x]);
                        r2[x] = row_of(j + 3, x);
                    }
                }
            }
        } else {
            // =========================================== softmax + epilogue
            // Warpgroup wg: heads 32 wg .. 32 wg + 31. A thread's lane of S^T
            // is key slot `slot_k`, low or high dims by `hi`; it takes the 16
            // heads from hb on, its partner 8 lanes away the others.
            const int wg = warp >> 2, q4 = warp & 3, h0 = 32 * wg, hi = (lane >> 3) & 1;
            const int hb = h0 + 16 * hi, slot_k = 16 * q4 + 8 * (lane >> 4) + (lane & 7);
            const uint32_t bar = 1 + wg;
            const uint32_t lane_addr = tmem + ((uint32_t)(32 * q4) << 16);
            const float sc = a.softmax_scale * kLog2e;
            bool ok = true, stop = false;
            for (int32_t i = 0; i < n_pieces && !stop; ++i, ++np) {
                const int32_t tt = ms->piece[i].t, nt = ms->piece[i].j1 - ms->piece[i].j0;
                const int32_t slot = ms->piece[i].slot;
                float lp[16], m_cur[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    lp[x] = 0.0f;
                    m_cur[x] = -INFINITY;
                }
                for (int32_t j = 0; j < nt; ++j, ++g) {
                    ok = cx.wait(&ms->kv_full[g & 1], (g >> 1) & 1, 30) &&
                         cx.wait(&ms->s_full[g & 1], (g >> 1) & 1, 31);
                    tc::tc_fence_after();
                    const bool key = (ms->valid[g & 1][q4 >> 1] >> (slot_k & 31)) & 1u;
                    float v[16];
                    auto load_scores = [&]() {
                        float lo[32], up[32];
                        const uint32_t addr = lane_addr + kColS + 128 * (g & 1) + h0;
                        tc::tmem_ld32(addr, lo);
                        tc::tmem_ld32(addr + 64, up);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            v[x] = (hi ? up[16 + x] : lo[x]) +
                                   __shfl_xor_sync(0xffffffffu, hi ? up[x] : lo[16 + x], 8);
                    };
                    load_scores();
                    // Scores in base 2 above the running maximum, which the
                    // first tile sets (its largest weight is then exactly 1 in
                    // bf16) and later ones move only when a score exceeds it
                    // by more than kLazyMax, so that O^T is rarely rescaled;
                    // the warpgroup agrees on it.
                    bool over = !ok || j == 0;
                    if (j > 0) {
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            v[x] = key ? fmaf(v[x], sc, -m_cur[x]) : -INFINITY;
                            over |= v[x] > kLazyMax;
                        }
                        over = bar_or(bar, over);
                    }
                    if (over) {
                        if (j > 0) {
                            ok = ok && cx.wait(&ms->kv_empty[(g - 1) & 1], ((g - 1) >> 1) & 1, 33);
                            tc::tc_fence_after();
                            load_scores();
                        }
                        if (!bar_and(bar, ok)) {
                            stop = true;
                            break;
                        }
#pragma unroll
                        for (int x = 0; x < 16; ++x) v[x] = key ? v[x] * sc : -INFINITY;
                        float(*red)[64] = ms->red[g & 1];
                        red[q4][hb + sum_index(lane)] = reduce_scatter16<true>(v, lane);
                        tc::named_bar_sync(bar, 128);
                        bool scale = false;
                        float al[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const float mt = fmaxf(fmaxf(red[0][hb + x], red[1][hb + x]),
                                                   fmaxf(red[2][hb + x], red[3][hb + x]));
                            const bool up = mt > m_cur[x] + kLazyMax;
                            al[x] = 1.0f;
                            if (up && m_cur[x] != -INFINITY) {
                                al[x] = tc::ex2_approx(m_cur[x] - mt);
                                scale = true;
                            }
                            if (up) m_cur[x] = mt;
                            lp[x] *= al[x];
                            v[x] = m_cur[x] == -INFINITY ? -INFINITY : v[x] - m_cur[x];
                        }
                        if (q4 == 0 && (lane & 23) == 0) {  // one lane for each 16 heads
#pragma unroll
                            for (int x = 0; x < 16; ++x) {
                                ms->m[hb + x] = m_cur[x];
                                ms->fac[hb + x] = al[x];
                            }
                        }
                        if (j > 0 && bar_or(bar, scale)) {
#pragma unroll 1
                            for (int d = 0; d < 4; ++d) {
                                float o[32];
                                const uint32_t addr = lane_addr + kColO + 64 * d + h0;
                                tc::tmem_ld32(addr, o);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int x = 0; x < 32; ++x) o[x] *= ms->fac[h0 + x];
                                tc::tmem_st32(addr, o);
                            }
                            tc::tmem_wait_st();
                        }
                    }
                    // weights (bf16) -> row of P^T: 32 bytes of its 128
                    unsigned char *prow = smem + kOffP + (g & 1) * 8192 + slot_k * 128;
#pragma unroll
                    for (int c8 = 0; c8 < 2; ++c8) {
                        uint32_t w4[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int x = 8 * c8 + 2 * y;
                            const float p0 = tc::ex2_approx(v[x]), p1 = tc::ex2_approx(v[x + 1]);
                            lp[x] += p0;
                            lp[x + 1] += p1;
                            const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
                            w4[y] = *reinterpret_cast<const uint32_t *>(&pb);
                        }
                        *reinterpret_cast<uint4 *>(prow + (((hb / 8 + c8) ^ (slot_k & 7)) << 4)) =
                            make_uint4(w4[0], w4[1], w4[2], w4[3]);
                    }
                    tc::fence_proxy_async_smem();
                    tc::tc_fence_before();
                    tc::mbar_arrive(&ms->p_full[g & 1]);
                }
                if (stop) break;
                // ---- row sums, then O^T
                float(*red)[64] = ms->red[g & 1];  // no step of this token reads it any more
                red[q4][hb + sum_index(lane)] = reduce_scatter16<false>(lp, lane);
                tc::named_bar_sync(bar, 128);
                if (q4 == 0) {
                    const int h = h0 + lane;
                    const float l = (red[0][h] + red[1][h]) + (red[2][h] + red[3][h]), m = ms->m[h];
                    float f = 1.0f;  // O^T times this
                    if (slot < 0) {
                        const float sk = a.sinks && h < a.H && ms->piece[i].k.seq >= 0
                                             ? __ldg(a.sinks + h) * kLog2e
                                             : -INFINITY;
                        const float M = fmaxf(m, sk);
                        const float w = m == -INFINITY ? 0.0f : tc::ex2_approx(m - M);
                        const float Z = fmaf(l, w, sk == -INFINITY ? 0.0f : tc::ex2_approx(sk - M));
                        f = Z > 0.0f ? w / Z : 0.0f;
                        if (a.lse && h < a.H)
                            a.lse[(int64_t)tt * a.H + h] = (M + tc::lg2_approx(Z)) * kLn2;
                    } else if (h < a.H) {
                        ws.m[slot * 64 + h] = m;
                        ws.l[slot * 64 + h] = l;
                    }
                    ms->fac[h] = f;
                }
                ok = cx.wait(&ms->o_full, np & 1, 32);
                if (!bar_and(bar, ok)) {
                    stop = true;
                    break;
                }
                tc::tc_fence_after();
                // Lane of O^T slab d: dim 64 d + lane of the low (q4 < 2) or the
                // high half, 32 heads a thread
                const int n_h = min(32, a.H - h0);
                const int dim = (q4 >> 1) * 256 + 32 * (q4 & 1) + lane;
                __nv_bfloat16 *outp = a.out + ((int64_t)tt * a.H + h0) * 512 + dim;
#pragma unroll 1
                for (int d = 0; d < 4; ++d) {
                    float o[32];
                    tc::tmem_ld32(lane_addr + kColO + 64 * d + h0, o);
                    tc::tmem_wait_ld();
                    if (d == 3) {  // O^T is read: the next token's may start
                        tc::tc_fence_before();
                        tc::mbar_arrive(&ms->o_empty);
                    }
                    if (slot >= 0) {
#pragma unroll
                        for (int x = 0; x < 32; x += 4)
                            if (x < n_h)
                                *ws.sums(slot, (h0 + x) >> 2, dim + 64 * d) =
                                    make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
                    } else {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (x < n_h)
                                outp[x * 512 + 64 * d] = __float2bfloat16_rn(o[x] * ms->fac[h0 + x]);
                    }
                }
                tc::named_bar_sync(bar, 128);  // fac, m and red are read
            }
        }
        __syncthreads();
        if (cx.aborted()) break;
    }

    // ------------------------------------------------------------- teardown
    if (warp == 8 || warp == 9) asm volatile("cp.async.wait_all;" ::: "memory");
    if (tid == 32 * kMmaWarp) {  // no copy outlives the CTA, no MMA its tensor memory
        if (nq > 0 && !tc::mbar_wait(&ms->q_full, (nq - 1) & 1)) cx.fail(26);
        if (issued) tc::mma_commit(&ms->drain);
        if (issued && !tc::mbar_wait(&ms->drain, 0)) cx.fail(24);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

// Block (c, y): heads 4 y .. 4 y + 3 of the token whose first tile CTA c held
// and that other CTAs went on with; two dims a thread. The first parts' sums
// are on their way before their factors are known.
constexpr int kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads)
sparse_mla_paged_join_kernel(const __grid_constant__ MlaPagedArgs a) {
    __shared__ float w_s[4][kMaxGrid];
    __shared__ float inv_s[4];
    const Space ws(a.workspace, a.H);
    grid_dependency_wait();
    launch_dependents();
    const Join jn = ws.join[blockIdx.x];
    if (jn.t < 0) return;
    const int quad = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t parts = jn.last - jn.first + 1;
    // slot of part i: the first CTA's second slot, then the others' first ones
    auto slot = [&](int32_t i) { return 2 * (jn.first + i) + (i == 0 ? 1 : 0); };
    constexpr int kB = 6;
    float4 v[kB][2];
    auto fetch = [&](int32_t i0) {
#pragma unroll
        for (int i = 0; i < kB; ++i)
            if (i0 + i < parts) {
                v[i][0] = *ws.sums(slot(i0 + i), quad, tid);
                v[i][1] = *ws.sums(slot(i0 + i), quad, tid + 256);
            }
    };
    fetch(0);
    const int h = 4 * quad + warp;
    if (warp < 4 && h < a.H) {  // one warp a head: the parts' factors
        const float sk = a.sinks ? __ldg(a.sinks + h) * kLog2e : -INFINITY;
        float m[(kMaxGrid + 31) / 32], l[(kMaxGrid + 31) / 32], M = sk;
#pragma unroll
        for (int i = 0; i < (kMaxGrid + 31) / 32; ++i) {
            const int32_t p = 32 * i + lane;
            m[i] = p < parts ? ws.m[slot(p) * 64 + h] : -INFINITY;
            l[i] = p < parts ? ws.l[slot(p) * 64 + h] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < (kMaxGrid + 31) / 32; ++i) M = fmaxf(M, m[i]);
        M = warp_max(M);
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < (kMaxGrid + 31) / 32; ++i) {
            const float f = m[i] == -INFINITY ? 0.0f : tc::ex2_approx(m[i] - M);
            if (32 * i + lane < parts) w_s[warp][32 * i + lane] = f;
            z = fmaf(l[i], f, z);
        }
        z = warp_sum(z) + (sk == -INFINITY ? 0.0f : tc::ex2_approx(sk - M));
        if (lane == 0) {
            inv_s[warp] = z > 0.0f ? 1.0f / z : 0.0f;
            if (a.lse) a.lse[(int64_t)jn.t * a.H + h] = (M + tc::lg2_approx(z)) * kLn2;
        }
    } else if (warp < 4) {
        for (int32_t p = lane; p < parts; p += 32) w_s[warp][p] = 0.0f;
        if (lane == 0) inv_s[warp] = 0.0f;
    }
    __syncthreads();
    float o[2][4] = {};
    for (int32_t i0 = 0; i0 < parts; i0 += kB) {
        if (i0 > 0) fetch(i0);
#pragma unroll
        for (int i = 0; i < kB; ++i)
            if (i0 + i < parts) {
                const float f[4] = {w_s[0][i0 + i], w_s[1][i0 + i], w_s[2][i0 + i], w_s[3][i0 + i]};
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    o[y][0] = fmaf(v[i][y].x, f[0], o[y][0]);
                    o[y][1] = fmaf(v[i][y].y, f[1], o[y][1]);
                    o[y][2] = fmaf(v[i][y].z, f[2], o[y][2]);
                    o[y][3] = fmaf(v[i][y].w, f[3], o[y][3]);
                }
            }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
        if (4 * quad + x < a.H) {
            __nv_bfloat16 *out = a.out + ((int64_t)jn.t * a.H + 4 * quad + x) * 512 + tid;
            out[0] = __float2bfloat16_rn(o[0][x] * inv_s[x]);
            out[256] = __float2bfloat16_rn(o[1][x] * inv_s[x]);
        }
}

}  // namespace

size_t mla_paged_workspace_bytes(int32_t T, int32_t H) {
    if (T <= 0) return 0;
    return kMaxGrid * sizeof(Join) +
           (size_t)2 * kMaxGrid * (2 * 64 + (size_t)(H + 3) / 4 * 4 * 512) * sizeof(float);
}

cudaError_t launch_sparse_mla_paged(MlaPagedArgs a, cudaStream_t stream) {
    static PerContext pc;
    int sms, dev;
    bool first;
    unsigned long long ctx;
    cudaError_t e = enter_context(pc, &sms, &first, &ctx, &dev);
    if (e != cudaSuccess) return e;
    if (first) {
        e = cudaFuncSetAttribute(sparse_mla_paged_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kSmemBytes);
        if (e != cudaSuccess) return e;
        entered_context(pc, dev, ctx);
    }
    CUtensorMap q_map;
    if (!encode_bf16_3d(&q_map, a.q, 512, a.H, a.T, 64, a.H, 1)) return cudaErrorInvalidValue;
    const int grid = min(sms, kMaxGrid);
    e = launch_early(sparse_mla_paged_kernel, dim3(grid), dim3(kThreads), kSmemBytes, stream, q_map, a);
    if (e != cudaSuccess) return e;
    return launch_early(sparse_mla_paged_join_kernel, dim3(grid, (a.H + 3) / 4),
                        dim3(kJoinThreads), 0, stream, a);
}

}  // namespace csa
