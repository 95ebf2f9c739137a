// Sparse MLA attention of new tokens over paged caches (sm_103a, tcgen05
// tensor cores, cp.async gathers): the keys of token t are the window rows of
// its sequence in the original-KV cache and the listed (or every visible) rows
// of the compressed cache, which holds them in bf16 or in 4 bits (q4.cuh).
//
//     l_i = scale q.kv_i ; Z = sum e^(l_i - m) + e^(sink - m)
//     out = sum e^(l_i - m) kv_i / Z ; lse = m + ln Z
//
// Work split. A token's keys form tiles of 64 slots. With no more tokens than
// CTAs, each token gets as many CTAs as its tiles need at the least number of
// tiles a CTA with which all parts fit the grid: long rows are spread over many
// CTAs and no CTA meets two tokens. With more, the tiles of all tokens, one
// after the other, are dealt to the CTAs in equal runs: a run covers the end of
// one token, whole tokens, and the start of one more. Whole tokens are finished
// in place; a CTA's one or two pieces of tokens go to its two slots of the
// workspace (fp32 sums with their running maximum), which the CTA that holds a
// token's first tile describes and a second kernel joins. The split follows
// from sizes and positions alone, so results repeat bit by bit.
//
// A tile. All heads share a row, which is both key and value, so a tile is
// loaded once for two products:
//     S = Q K^T: heads x keys, K = 512. 64 heads fill half of M = 128, which
//          costs the tensor core as much as all of it, so the other half of M
//          takes the heads' dims 256-511 and N = 128 the keys' low and high
//          dims: 16 MMAs in place of 32. Of the four blocks of the result the
//          two matching ones are added; rows of the low and the high half
//          alternate in groups of 8, so a head's two partial scores sit 8
//          lanes apart in one warp. Q is the operand
//          in tensor memory (128 columns), which leaves shared memory to
//          three tiles; a token's Q comes through the tiles' stages like one.
//     O^T += V^T P^T: 4 slabs of 128 dims x 64 heads, K = 64 keys; V is the
//          K tile's bytes read MN-major. P is rounded to bf16, V's type, as in
//          the packed forward; its sums stay fp32. The output is then off by
//          up to 2.15e-3 (norm of the error over the norm, normal inputs),
//          where rounding the output alone gives 1.66e-3. With the rounded-off
//          part of P as a second bf16 operand it was 1.66e-3 too, but that
//          takes 16 more MMAs a tile: one token 12.8 -> 13.5 us, 64 tokens
//          26.4 -> 28.8, 81 drafted 33.2 -> 37.0, long rows 59.9 -> 70.9 (68.9
//          by the MMAs alone). Rounding was kept.
// Shared memory holds three tiles (192 KB) and two P (16 KB); tensor memory Q
// (128 columns), S (128) and O^T (256). The scores of the next tile are
// computed while this one's softmax runs. Rows are gathered by cp.async; their
// pages are found some tiles ahead by a warp of its own.
//
// Bound by HBM with long rows, by the latency of its steps with few tiles a
// CTA. With 64 heads, join included: one token of 640 keys 12.8 us, 64 of them
// 26.4 us, six long rows (225 MB read) 59.9 us or 3.8 TB/s.
//
// Compressed rows in 4 bits (Q4). The window's slots are padded to whole tiles,
// so that a tile is of one kind. A tile of 4-bit rows comes to shared memory as
// it is (24 KB, three on their way) and eight more warps turn it into a bf16
// tile, of which two fit beside them; what follows is as above, over values
// that bf16 holds exactly. The same cases: one token 14.6 us, 64 tokens 29.0,
// long rows (85 MB read) 71.1 or 1.2 TB/s. Long rows are bound by a tile's way
// through the two stages: turning it 2000 clocks beside the softmax (1320 by
// itself), scores 1400 and 650 until they are seen, softmax 1400, O^T 830 and
// 390; the tensor core is busy a quarter of the time. Measured on the way and
// dropped, long rows: a bulk copy a row 100 us; the turning unrolled, four warps
// of it 105, as a loop 73; stages filled and given back in quarters 89; codes
// prefetched into registers in place of raw tiles, with three bf16 stages 74 to
// 81; scores and O^T issued by two warps 71.2; that over tiles of 32 keys, four
// stages and scores twice buffered 70.0 (64 tokens 29.3).
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "q4.cuh"
#include "tc_ptx.cuh"

namespace csa {

namespace {

constexpr int kTile = 64;
constexpr int kMaxGrid = 160;     // CTAs of the persistent grid (sizes the workspace)
constexpr int kRing = 4;          // tiles whose rows are found ahead of the loaders
constexpr int kPieces = 64;       // pieces of a run described in shared memory at a time
constexpr float kLazyMax = 8.0f;  // base-2 units
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// shared memory map (offsets from a 1024-byte aligned base)
constexpr uint32_t kStage = 65536;  // 4 dim groups x 8 x [low, high] x [8 keys x 128 B]
constexpr uint32_t kRawTile = kTile * q4::kRow;  // rows as they are, each line of 128 bytes swizzled

// Tokens whose tiles are counted in one scan, whatever the block's threads: a
// token has up to kMaxKeys slots in either cache, and their sum takes 32 bits.
constexpr int kScan = 384;
static_assert((int64_t)kScan * 2 * (kMaxKeys / kTile) <= INT32_MAX, "a scan's sum");

constexpr int kLoaders = 64;
constexpr int kMmaWarp = 10;
constexpr int kFindWarp = 11;

// Both forms of compressed rows: Q4 false, bf16; true, 4 bits.
template <bool Q4>
struct Form {
    // 8 softmax and epilogue warps, 2 loaders, 1 MMA, 1 look-up; with 4-bit rows
    // 8 more that turn them into bf16
    static constexpr int kSpreadWarps = Q4 ? 8 : 0;
    static constexpr int kThreads = 384 + 32 * kSpreadWarps;
    static constexpr int kStages = Q4 ? 2 : 3;  // tiles in bf16
    static constexpr int kRaw = Q4 ? 3 : 0;     // tiles of 4-bit rows on their way
    static constexpr uint32_t kOffP = kStages * kStage;  // 2 x [64 heads x 64 keys] bf16, K-major
    static constexpr uint32_t kOffRaw = kOffP + 16384;
    static constexpr uint32_t kOffMisc = kOffRaw + kRaw * kRawTile;
};

// tensor memory columns
constexpr uint32_t kColQ = 0;    // [low, high] heads x 256 dims, two a column
constexpr uint32_t kColS = 128;  // [low, high] heads x [low, high] keys
constexpr uint32_t kColO = 256;  // 4 slabs of 128 d x 64 heads
constexpr uint32_t kTmemCols = 512;

struct Join {
    int32_t t, first, last, pad;  // token t is spread over CTAs first..last
};
// Join entries: one a token while there are no more tokens than CTAs, else one
// a CTA, of the token that starts in it and goes on in others.

// Workspace: Join [kMaxGrid], then (m, l) [2 kMaxGrid][64], then the sums
// [2 kMaxGrid][ceil(H / 4)][512][4 heads]: a thread of the epilogue holds one
// dim of 32 heads, so a warp writes 512 bytes at once.
struct Space {
    Join *join;
    float2 *ml;
    float *o;
    int32_t quads;
    __host__ __device__ Space(void *p, int32_t H) {
        join = static_cast<Join *>(p);
        ml = reinterpret_cast<float2 *>(join + kMaxGrid);
        o = reinterpret_cast<float *>(ml + 2 * kMaxGrid * 64);
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
    int32_t win_slots;  // of n_win rows: with 4-bit rows whole tiles, so that a tile is of one kind
    __device__ __forceinline__ uint32_t slots() const { return (uint32_t)win_slots + (uint32_t)n_cmp; }
    __device__ __forceinline__ int32_t tiles() const {  // a token without keys has one, empty
        return max(1, (int32_t)((slots() + kTile - 1) / kTile));
    }
};

template <bool Q4>
__device__ __forceinline__ Keys token_keys(const MlaPagedArgs &a, int32_t t, bool report) {
    Keys k = {-1, 0, 0, 0, 0, 0};
    const int32_t pos = __ldg(a.q_pos + t);
    const int32_t b = paged_seq(a.q_seq, a.batch, t, pos);
    if (b < 0) {
        if (b == -2 && report) report_error(a.err, kErrCheck, kKerMlaPaged, 1);
        return k;
    }
    k.seq = b;
    k.win_start = max(pos - a.window + 1, 0);
    k.n_win = pos - k.win_start + 1;
    k.win_slots = Q4 ? (k.n_win + kTile - 1) / kTile * kTile : k.n_win;
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
    if (i < (uint32_t)k.win_slots || i >= k.slots()) return -1;
    const int32_t e = (int32_t)(i - (uint32_t)k.win_slots);
    return a.idx ? __ldg(a.idx + (int64_t)t * a.topk + e) : e;
}

__device__ __forceinline__ Slot slot_page(const MlaPagedArgs &a, const Keys &k, uint32_t i, int32_t row) {
    const bool win = i < (uint32_t)k.win_slots;
    if (row < 0 || (!win && row >= k.vis)) return {-1, -1, win};
    const PagedRows &p = win ? a.ori : a.cmp;
    const uint32_t pg = (uint32_t)row / (uint32_t)p.page_size;
    const int32_t in = row - (int32_t)pg * p.page_size;
    return {in, pg < (uint32_t)p.max_pages ? __ldg(p.pages + (int64_t)k.seq * p.max_pages + pg) : -1, win};
}

// nullptr: no key, or its page is evicted or absent (recorded). Window rows are
// never evicted by weight: their table's mark is an absent page. Rows of the
// compressed cache may be of 384 bytes: the caller knows the slot's kind.
template <bool Q4>
__device__ __forceinline__ const __nv_bfloat16 *slot_ptr(const MlaPagedArgs &a, const Slot &s) {
    if (s.in < 0) return nullptr;
    const PagedRows &p = s.win ? a.ori : a.cmp;
    if ((uint32_t)s.phys >= (uint32_t)p.num_pages) {
        if (s.win || s.phys != CSA_PAGE_EVICTED) report_error(a.err, kErrCheck, kKerMlaPaged, 3);
        return nullptr;
    }
    const int64_t row = (int64_t)s.phys * p.page_size + s.in;
    return p.base + row * (Q4 && !s.win ? q4::kRow / 2 : 512);
}

// A stretch of tiles [j0, j1) of one token, worked by one CTA.
struct Piece {
    int32_t t, j0, j1;
    int32_t slot;  // workspace slot, or -1: the whole token
    Keys k;
};

template <bool Q4>
struct Misc {
    static constexpr int kStages = Form<Q4>::kStages;
    uint64_t q_full;
    uint64_t kv_full[kStages], kv_empty[kStages];
    uint64_t raw_full[Q4 ? 3 : 1], raw_empty[Q4 ? 3 : 1];
    uint64_t s_full, s_empty, p_full[2];
    uint64_t o_full, o_empty, drain;
    uint64_t ring_full[kRing], ring_empty[kRing];
    const __nv_bfloat16 *ring[kRing][kTile];  // pool rows of a tile's slots, nullptr: no key
    uint32_t tmem_base;
    int32_t abort;
    int64_t run_s, run_e;  // the CTA's run of tiles, of `per` each
    int64_t per;
    int64_t run_base;      // tiles before token run_t
    int64_t done;          // tiles up to the end of the batch
    int32_t run_t;         // token holding the CTA's next tile
    int32_t n_pieces;
    int32_t tiles[kMaxGrid];  // of each token, with no more tokens than CTAs
    int32_t scan[Form<Q4>::kThreads / 32 + 1];
    uint32_t valid[kStages][2];  // per stage and loader warp: 32 slot bits
    uint32_t raw_valid[Q4 ? 3 : 1][2];
    Piece piece[kPieces];
    float red[2][2][64];       // [tile parity][warpgroup][head]
    alignas(16) float fac[64];  // a rescaling's or the epilogue's factor
};

template <bool Q4>
constexpr size_t smem_bytes() {
    return Form<Q4>::kOffMisc + sizeof(Misc<Q4>) + 1024;
}
static_assert(smem_bytes<false>() <= 232448 && smem_bytes<true>() <= 232448, "shared memory budget");
static_assert(Form<true>::kRaw == 3, "barriers of the raw tiles");

// AND / OR of v over the 256 softmax threads.
__device__ __forceinline__ bool all_of(bool v) {
    uint32_t out;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(out)
        : "r"((uint32_t)v)
        : "memory");
    return out != 0;
}
__device__ __forceinline__ bool any_of(bool v) { return !all_of(!v); }

// D += A B with A in tensor memory (lane = row, two bf16 of K a column).
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// N columns (16 or 32) of tensor memory.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[N]) {
    if constexpr (N == 16) tc::tmem_ld16(taddr, v);
    else tc::tmem_ld32(taddr, v);
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&v)[N]) {
    if constexpr (N == 16) tc::tmem_st16(taddr, v);
    else tc::tmem_st32(taddr, v);
}

// Of a piece's tiles, Q being the first, the number of the first with 4-bit rows.
__device__ __forceinline__ int32_t first_coded(const Piece &p) {
    return 1 + max(p.k.win_slots / kTile - p.j0, 0);
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(tc::smem_u32(bar)), "r"(n) : "memory");
}

// A warp's eight rows of a raw tile, to bf16 in a stage. Lane: row `lane % 8`
// and of its 14 pieces of 32 codes (16 bytes) every fourth; in the
// last round half the lanes copy the rotary dims. Eight lanes read and write
// eight rows, at eight places of a swizzled line: no bank conflicts. A row of
// zeros (no key) gives zeros. The loops stay loops: every role runs its own code
// on the same SM, and its instructions have to be fetched.
__device__ __forceinline__ void spread_rows(const unsigned char *raw, unsigned char *stage, int w, int lane) {
    const int r = lane & 7, k = lane >> 3;
    raw += (8 * w + r) * q4::kRow;
    stage += w * 2048 + r * 128;
    const float unit = q4::pow2((int)raw[q4::kExp ^ (r << 4)] - 127);
    auto put = [&](int piece, const uint4 &c) {  // 32 dims
        const float2 f =
            q4::scales2(*reinterpret_cast<const uint16_t *>(raw + ((q4::kScales + 2 * piece) ^ (r << 4))));
        const __nv_bfloat162 s0 = q4::scale_pair(f.x, unit), s1 = q4::scale_pair(f.y, unit);
        unsigned char *line = stage + ((piece & 7) >> 1) * 16384 + (piece >> 3) * 1024;
        const uint32_t word[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4 *>(line + (((4 * (piece & 1) + x) ^ r) << 4)) =
                q4::eight(word[x], x < 2 ? s0 : s1);
    };
    uint4 c = *reinterpret_cast<const uint4 *>(raw + ((16 * k) ^ (r << 4)));
#pragma unroll 1
    for (int piece = k; piece < 12; piece += 4) {
        const uint4 now = c;
        c = *reinterpret_cast<const uint4 *>(raw + ((16 * (piece + 4)) ^ (r << 4)));
        put(piece, now);
    }
    if (k < 2) {
        put(12 + k, c);
    } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4 *>(stage + 3 * 16384 + 1024 + (((4 * (k - 2) + x) ^ r) << 4)) =
                *reinterpret_cast<const uint4 *>(raw + ((q4::kTail + 64 * (k - 2) + 16 * x) ^ (r << 4)));
    }
}

template <bool Q4>
__global__ void __launch_bounds__(Form<Q4>::kThreads, 1)
sparse_mla_paged_kernel(const __grid_constant__ MlaPagedArgs a) {
    using F = Form<Q4>;
    constexpr int kThreads = F::kThreads, kStages = F::kStages, kSpreadWarps = F::kSpreadWarps;
    constexpr int kRaw = Q4 ? F::kRaw : 1;
    constexpr uint32_t kOffP = F::kOffP;
    constexpr int kCols = Q4 ? 16 : 32;  // tensor memory columns a thread takes at a time: its registers
    using Misc = Misc<Q4>;
    using Ctx = PipeWaits<Misc, kKerMlaPaged>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc *ms = reinterpret_cast<Misc *>(smem + F::kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Space ws(a.workspace, a.H);
    const Ctx cx{ms, a.err, a.wait_ns};
    const int32_t c = blockIdx.x;

    if (tid == 0) {
        tc::mbar_init(&ms->q_full, 256);
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&ms->kv_full[i], Q4 ? 33 * kSpreadWarps : kLoaders + 2);
            tc::mbar_init(&ms->kv_empty[i], 1);
        }
        tc::mbar_init(&ms->s_full, 1);
        tc::mbar_init(&ms->s_empty, 256);
        for (int i = 0; i < 2; ++i) tc::mbar_init(&ms->p_full[i], 256);
        tc::mbar_init(&ms->o_full, 1);
        tc::mbar_init(&ms->o_empty, 256);
        tc::mbar_init(&ms->drain, 1);
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(&ms->ring_full[i], 32);
            tc::mbar_init(&ms->ring_empty[i], kLoaders + 32 * kSpreadWarps);
        }
        for (int i = 0; Q4 && i < kRaw; ++i) {
            tc::mbar_init(&ms->raw_full[i], kLoaders + 2);
            tc::mbar_init(&ms->raw_empty[i], kSpreadWarps);
        }
        ms->abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&ms->tmem_base, kTmemCols);
        tc::tmem_relinquish();
    }
    // everything above is local: wait for the kernels before this one
    grid_dependency_wait();
    launch_dependents();
    const bool by_token = a.T <= (int32_t)gridDim.x;  // at most kMaxGrid, and a thread for each
    if (tid == 0 && !by_token) ws.join[c] = {-1, 0, 0, 0};
    // The lists and tables, when a line each for the grid's threads covers
    // them, are on their way to L2 while the runs are worked out.
    {
        const int64_t line = (int64_t)c * kThreads + tid, lines = (int64_t)gridDim.x * kThreads;
        auto send_for = [&](const int32_t *p, int64_t n) {
            const int64_t bytes = n * 4;
            if (p && bytes <= lines * 128 && line * 128 < bytes)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char *>(p) + line * 128));
        };
        send_for(a.idx, (int64_t)a.T * a.topk);
        send_for(a.ori.pages, (int64_t)a.batch * a.ori.max_pages);
        if (a.cmp.base) send_for(a.cmp.pages, (int64_t)a.batch * a.cmp.max_pages);
    }
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();

    // ---------------------------------------------- this CTA's share of tiles
    // (What only the batches below need waits in shared memory: every role's
    // code would carry it in registers.)
    if (by_token) {
        Keys k = {-1, 0, 0, 0, 0, 0};
        int32_t n = 0;
        if (tid < a.T) {
            k = token_keys<Q4>(a, tid, c == 0);
            n = k.tiles();
            ms->tiles[tid] = n;
        }
        __syncthreads();
        tc::tc_fence_after();
        // Every warp finds the least number of tiles a CTA may get so that the
        // tokens' parts fit the grid, and with it this CTA's token and part.
        // (Loops over rows of 32 tokens, not unrolled: code that runs once costs
        // more to fetch than to execute.)
        const int rows = (a.T + 31) >> 5;
        auto tiles_at = [&](int i) { return 32 * i + lane < a.T ? ms->tiles[32 * i + lane] : 0; };
        auto parts_of = [&](int32_t x, int32_t q) { return ((uint32_t)x + (uint32_t)q - 1u) / (uint32_t)q; };
        int32_t most = 1;
        int64_t N = 0;
#pragma unroll 1
        for (int i = 0; i < rows; ++i) {
            const int32_t x = tiles_at(i);
            most = max(most, x);
            N += ((int64_t)__reduce_add_sync(0xffffffffu, (uint32_t)x >> 16) << 16) +
                 __reduce_add_sync(0xffffffffu, (uint32_t)x & 0xffffu);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        const int32_t G = gridDim.x;
        int32_t lo = (int32_t)div64(N + G - 1, G), up = most;  // N / q + T <= G suffices
        if (G > a.T) up = (int32_t)min((int64_t)most, div64(N, G - a.T) + 1);
#pragma unroll 1
        while (lo < up) {
            const int32_t q = lo + (up - lo) / 2;
            uint32_t parts = 0;
#pragma unroll 1
            for (int i = 0; i < rows; ++i) parts += parts_of(tiles_at(i), q);
            if (__reduce_add_sync(0xffffffffu, parts) <= (uint32_t)G) up = q;
            else lo = q + 1;
        }
        int32_t mine_t = -1, mine_first = 0, mine_parts = 0, before = 0;
#pragma unroll 1
        for (int i = 0; i < rows && before <= c; ++i) {
            const int32_t p = (int32_t)parts_of(tiles_at(i), lo);
            int32_t x = p;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            const int32_t first = before + x - p;
            if (first <= c && c < first + p) {
                mine_t = 32 * i + lane;
                mine_first = first;
                mine_parts = p;
            }
            before += __shfl_sync(0xffffffffu, x, 31);
        }
        const uint32_t who = __ballot_sync(0xffffffffu, mine_t >= 0);
        if (who == 0) {  // no part left for this CTA
            __syncthreads();
            if (warp == kMmaWarp) tc::tmem_dealloc(ms->tmem_base, kTmemCols);
            return;
        }
        const int src = __ffs(who) - 1;
        const int32_t t = __shfl_sync(0xffffffffu, mine_t, src);
        const int32_t first = __shfl_sync(0xffffffffu, mine_first, src);
        const int32_t parts = __shfl_sync(0xffffffffu, mine_parts, src);
        if (tid == t) {
            const uint32_t part = (uint32_t)(c - first);
            ms->piece[0] = {t, (int32_t)(part * (uint32_t)n / (uint32_t)parts),
                            (int32_t)((part + 1u) * (uint32_t)n / (uint32_t)parts),
                            parts == 1 ? -1 : 2 * c + (part == 0 ? 1 : 0), k};
            if (part == 0) ws.join[t] = {t, first, first + parts - 1, 0};
            ms->n_pieces = 1;
            ms->done = ms->run_e = 1;
        }
    } else {
        // Equal runs. Tokens are scanned kScan at a time: once to count the
        // tiles, once for the token that holds the run's first one.
        auto tiles_of = [&](int32_t t, bool report) {
            return tid < kScan && t < a.T ? token_keys<Q4>(a, t, report).tiles() : 0;
        };
        int64_t N = 0;
        int32_t total;
        for (int32_t t0 = 0; t0 < a.T; t0 += kScan) {
            block_exclusive_scan<kThreads>(tiles_of(t0 + tid, c == 0), ms->scan, &total);
            N += total;
        }
        tc::tc_fence_after();
        const int64_t per = div64(N + gridDim.x - 1, gridDim.x);
        const int64_t s = min(c * per, N), e = min(s + per, N);
        if (tid == 0) {
            ms->run_s = s;
            ms->run_e = e;
            ms->per = per;
        }
        if (s == e) {  // no run left for this CTA
            __syncthreads();
            if (warp == kMmaWarp) tc::tmem_dealloc(ms->tmem_base, kTmemCols);
            return;
        }
        int64_t base = 0;
        for (int32_t t0 = 0; t0 < a.T && base <= s; t0 += kScan) {
            const int32_t t = t0 + tid, nt = tiles_of(t, false);
            const int64_t bt = base + block_exclusive_scan<kThreads>(nt, ms->scan, &total);
            if (bt <= s && s < bt + nt) {
                ms->run_t = t;
                ms->run_base = bt;
            }
            base += total;
        }
    }
    __syncthreads();
    const uint32_t tmem = ms->tmem_base;

    // counters of each role, kept across batches of pieces
    uint32_t g = 0, np = 0;
    uint32_t rc = 0;  // raw tiles so far
    bool issued = false;
    do {
        // ------------------------------------------------- a batch of pieces
        if (!by_token) {
            const int32_t t_first = ms->run_t, t = t_first + tid;
            const int64_t base = ms->run_base, s = ms->run_s, e = ms->run_e;
            int32_t total, n = 0;
            Keys k = {-1, 0, 0, 0, 0, 0};
            if (tid < kPieces && t < a.T) {
                k = token_keys<Q4>(a, t, false);
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
                    ws.join[c] = {t, c, (int32_t)div64(b + n - 1, ms->per), 0};
                if (tid == kPieces - 1 || t + 1 == a.T || b + n >= e) {
                    ms->n_pieces = tid + 1;
                    ms->done = min(e, b + n);
                }
            }
            if (tid == 0) {
                ms->run_t = t_first + kPieces;
                ms->run_base = base + total;
            }
        }
        __syncthreads();
        const int32_t n_pieces = ms->n_pieces;

        if (warp == kMmaWarp) {
            // ===================================================== MMA warp
            if (lane == 0) {
                constexpr uint32_t id_s = tc::idesc_bf16(128, 128, false, false);
                constexpr uint32_t id_o = tc::idesc_bf16(128, 64, true, false);
                const uint64_t ds_b = tc::smem_desc(tc::smem_u32(smem), 16, 1024);
                const uint64_t do_a = tc::smem_desc(tc::smem_u32(smem), 1024, 2048);
                const uint64_t do_b = tc::smem_desc(tc::smem_u32(smem + kOffP), 16, 1024);
                bool ok = true;
                for (int32_t i = 0; i < n_pieces && ok; ++i, ++np) {
                    const int32_t nt = ms->piece[i].j1 - ms->piece[i].j0;
                    ++g;  // the stage of Q
                    if (!(ok = cx.wait(&ms->q_full, np & 1, 20))) break;
                    // O^T of tile jo and scores of tile js, whichever is ready
                    // first, O^T before scores: it frees a stage, and the load
                    // that follows is the longest part of a tile's way.
                    int32_t js = 0, jo = 0;
                    const uint32_t k0 = g - np - 1;  // key tiles before this piece
                    uint64_t since = 0;
                    while (jo < nt) {
                        const uint32_t xs = k0 + js, xo = k0 + jo;  // key tiles
                        const uint32_t gs = g + js, go = g + jo;    // their stages
                        if (jo < js && tc::mbar_try_wait(&ms->p_full[xo & 1], (xo >> 1) & 1, 20)) {
                            if (jo == 0 && !(ok = cx.wait(&ms->o_empty, (np & 1) ^ 1, 23))) break;
                            tc::tc_fence_after();
                            const uint32_t st = (go % kStages) * kStage, pb = (xo & 1) * 8192;
#pragma unroll
                            for (int d = 0; d < 4; ++d)
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    tc::mma_bf16(tmem + kColO + 64 * d,
                                                 tc::desc_add(do_a, st + d * 16384 + kk * 4096),
                                                 tc::desc_add(do_b, pb + kk * 32), id_o, (jo | kk) != 0);
                            tc::mma_commit(&ms->kv_empty[go % kStages]);
                            ++jo;
                            since = 0;
                            continue;
                        }
                        // js <= jo + 1: P of tile js goes where P of tile js - 2 was
                        if (js < nt && js <= jo + 1 &&
                            tc::mbar_try_wait(&ms->kv_full[gs % kStages], (gs / kStages) & 1, 20) &&
                            (xs == 0 || tc::mbar_try_wait(&ms->s_empty, (xs - 1) & 1, 20))) {
                            tc::fence_proxy_async_smem();  // cp.async wrote through the generic proxy
                            tc::tc_fence_after();
                            const uint32_t st = (gs % kStages) * kStage;
#pragma unroll
                            for (int d = 0; d < 4; ++d)
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    mma_bf16_ta(tmem + kColS, tmem + kColQ + 8 * (4 * d + kk),
                                                tc::desc_add(ds_b, st + d * 16384 + kk * 32), id_s,
                                                (d | kk) != 0);
                            issued = true;
                            tc::mma_commit(&ms->s_full);
                            ++js;
                            since = 0;
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
                    g += nt;
                    tc::mma_commit(&ms->o_full);
                }
            }
            __syncwarp();
        } else if (warp == 8 || warp == 9) {
            // ================================================= loader warps
            // Warp w copies rows 32 w .. 32 w + 31 of every tile.
            const int w = warp - 8;
            bool ok = true;
            for (int32_t i = 0; i < n_pieces && ok; ++i) {
                const int32_t nt = 1 + ms->piece[i].j1 - ms->piece[i].j0;  // Q, then the keys
                const int32_t coded = Q4 ? first_coded(ms->piece[i]) : nt;
                for (int32_t j = 0; j < nt; ++j, ++g) {
                    ok = __all_sync(0xffffffffu,
                                    cx.wait(&ms->ring_full[g % kRing], (g / kRing) & 1, 40));
                    if (!ok) break;
                    const __nv_bfloat16 *mine = ms->ring[g % kRing][32 * w + lane];
                    tc::mbar_arrive(&ms->ring_empty[g % kRing]);
                    const uint32_t m = __ballot_sync(0xffffffffu, mine != nullptr), st = g % kStages;
                    if constexpr (Q4) {
                        // Tiles in bf16 are the spread warps', which follow the
                        // stages one by one. Four rows of 384 bytes are three
                        // instructions. (A bulk copy a row took 65 clocks to
                        // issue, 4200 a tile.)
                        if (j < coded) continue;
                        const uint32_t rs = rc % kRaw;
                        ok = __all_sync(0xffffffffu, cx.wait(&ms->raw_empty[rs], ((rc / kRaw) & 1) ^ 1, 42));
                        if (!ok) break;
                        ++rc;
                        const uint32_t raw = tc::smem_u32(smem + F::kOffRaw + rs * kRawTile) + 32 * w * q4::kRow;
#pragma unroll 1
                        for (int x = 0; x < 3; ++x) {
                            const int sub = (32 * x + lane) / 24, piece = (32 * x + lane) % 24;
#pragma unroll
                            for (int r = 0; r < 32; r += 4) {
                                const unsigned char *src = reinterpret_cast<const unsigned char *>(
                                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), r + sub));
                                const uint32_t bytes = src ? 16u : 0u;  // no key: zeros
                                if (!src) src = reinterpret_cast<const unsigned char *>(a.q);
                                cp_async16(raw + (r + sub) * q4::kRow + (16 * piece ^ (((r + sub) & 7) << 4)),
                                           src + 16 * piece, bytes);
                            }
                        }
                        cp_async_arrive(&ms->raw_full[rs]);
                        if (lane == 0) {
                            ms->raw_valid[rs][w] = m;
                            tc::mbar_arrive(&ms->raw_full[rs]);
                        }
                        continue;
                    }
                    ok = __all_sync(0xffffffffu, cx.wait(&ms->kv_empty[st], ((g / kStages) & 1) ^ 1, 41));
                    if (!ok) break;
                    // Half a row (512 bytes) an instruction: pieces of 128 bytes
                    // of several rows took twice as long to issue. Lane: dim
                    // group lane / 8, 16-byte unit lane % 8 of its 128 bytes.
                    const uint32_t stage =
                        tc::smem_u32(smem + st * kStage) + (lane >> 3) * 16384 + w * 4 * 2048;
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
                    cp_async_arrive(&ms->kv_full[st]);
                    if (lane == 0) {
                        ms->valid[st][w] = m;
                        tc::mbar_arrive(&ms->kv_full[st]);
                    }
                }
            }
        } else if (Q4 && warp > kFindWarp) {
            // ================================================= spread warps
            // Warp w: rows 8 w .. 8 w + 7 of every tile, from a raw tile or, in
            // bf16, from global memory. (kv_full: 33 arrivals a warp, one of
            // each lane's copies and one more, or all at once.)
            const int w = warp - kFindWarp - 1;
            bool ok = true;
            for (int32_t i = 0; i < n_pieces && ok; ++i) {
                const int32_t nt = 1 + ms->piece[i].j1 - ms->piece[i].j0, coded = first_coded(ms->piece[i]);
                for (int32_t j = 0; j < nt; ++j, ++g) {
                    const uint32_t st = g % kStages, rs = rc % kRaw;
                    ok = __all_sync(0xffffffffu, cx.wait(&ms->ring_full[g % kRing], (g / kRing) & 1, 45));
                    if (!ok) break;
                    const __nv_bfloat16 *mine = ms->ring[g % kRing][32 * (w >> 2) + lane];
                    tc::mbar_arrive(&ms->ring_empty[g % kRing]);
                    ok = __all_sync(0xffffffffu,
                                    cx.wait(&ms->kv_empty[st], ((g / kStages) & 1) ^ 1, 43) &&
                                        (j < coded || cx.wait(&ms->raw_full[rs], (rc / kRaw) & 1, 44)));
                    if (!ok) break;
                    if (j < coded) {
                        const uint32_t m = __ballot_sync(0xffffffffu, mine != nullptr);
                        const uint32_t stage = tc::smem_u32(smem + st * kStage) + (lane >> 3) * 16384 + w * 2048;
#pragma unroll 2
                        for (int r = 0; r < 8; ++r) {
                            const __nv_bfloat16 *src = reinterpret_cast<const __nv_bfloat16 *>(__shfl_sync(
                                0xffffffffu, reinterpret_cast<unsigned long long>(mine), 8 * (w & 3) + r));
                            const uint32_t bytes = src ? 16u : 0u;  // no key: zeros
                            if (!src) src = a.q;
                            const uint32_t dst = stage + r * 128 + (((lane ^ r) & 7) << 4);
                            cp_async16(dst, src + lane * 8, bytes);
                            cp_async16(dst + 1024, src + 256 + lane * 8, bytes);
                        }
                        cp_async_arrive(&ms->kv_full[st]);
                        if (lane == 0) {
                            if ((w & 3) == 0) ms->valid[st][w >> 2] = m;
                            tc::mbar_arrive(&ms->kv_full[st]);
                        }
                        continue;
                    }
                    ++rc;
                    if (lane == 0 && (w & 3) == 0) ms->valid[st][w >> 2] = ms->raw_valid[rs][w >> 2];
                    spread_rows(smem + F::kOffRaw + rs * kRawTile, smem + st * kStage, w, lane);
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive_n(&ms->kv_full[st], 33);
                        tc::mbar_arrive(&ms->raw_empty[rs]);
                    }
                }
            }
        } else if (warp == kFindWarp) {
            // ================================================= look-up warp
            // Two slots a lane. While a tile's rows are handed to the loaders,
            // the pages of the next tile and the list entries of the one after
            // it are being read. (Sending for the rows themselves ahead of
            // their copies, by L2 prefetches, made long rows 15 % slower.)
            bool ok = true;
            for (int32_t i = 0; i < n_pieces && ok; ++i) {
                const int32_t tt = ms->piece[i].t, j0 = ms->piece[i].j0, j1 = ms->piece[i].j1;
                const Keys kt = ms->piece[i].k;
                auto at = [&](int32_t j, int x) { return (uint32_t)j * kTile + 32 * x + lane; };
                auto row_of = [&](int32_t j, int x) { return j < j1 ? slot_row(a, kt, tt, at(j, x)) : -1; };
                // Q first: heads past H are zero rows
                ok = __all_sync(0xffffffffu, cx.wait(&ms->ring_empty[g % kRing], ((g / kRing) & 1) ^ 1, 51));
                if (!ok) break;
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    ms->ring[g % kRing][32 * x + lane] =
                        32 * x + lane < a.H ? a.q + ((int64_t)tt * a.H + 32 * x + lane) * 512 : nullptr;
                tc::mbar_arrive(&ms->ring_full[g % kRing]);
                ++g;
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
#pragma unroll
                    for (int x = 0; x < 2; ++x) ms->ring[g % kRing][32 * x + lane] = slot_ptr<Q4>(a, s0[x]);
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
            // A thread's lane of S is head `h`, low or high dims by `hi`; of
            // the 32 keys of its warpgroup wg it takes 16, its
            // partner 8 lanes away the others.
            const int wg = warp >> 2, q4 = warp & 3, hi = (lane >> 3) & 1;
            const int h = 16 * q4 + 8 * (lane >> 4) + (lane & 7);
            const uint32_t lane_addr = tmem + ((uint32_t)(32 * q4) << 16);
            const float sc = a.softmax_scale * kLog2e;
            // Q of the piece whose stage is next, to tensor memory: this
            // thread's row is dims 256 hi .. + 255 of head h, its warpgroup's
            // half of the columns.
            auto take_q = [&]() -> bool {
                if (!all_of(cx.wait(&ms->kv_full[g % kStages], (g / kStages) & 1, 34))) return false;
                const unsigned char *q = smem + (g % kStages) * kStage + 2 * wg * 16384 + (h >> 3) * 2048 +
                                         hi * 1024 + (h & 7) * 128;
#pragma unroll
                for (int d = 0; d < 64; d += kCols) {
                    float v[kCols];  // the bits as they are
#pragma unroll
                    for (int u = 0; u < kCols / 4; ++u) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(
                            q + (d >> 5) * 16384 + (((u + (d & 31) / 4) ^ (h & 7)) << 4));
                        v[4 * u] = __uint_as_float(x.x);
                        v[4 * u + 1] = __uint_as_float(x.y);
                        v[4 * u + 2] = __uint_as_float(x.z);
                        v[4 * u + 3] = __uint_as_float(x.w);
                    }
                    tmem_st<kCols>(lane_addr + kColQ + 64 * wg + d, v);
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                tc::mbar_arrive(&ms->q_full);
                tc::named_bar_sync(1, 256);
                if (tid == 0) tc::mbar_arrive(&ms->kv_empty[g % kStages]);
                ++g;
                return true;
            };
            bool ok = true, stop = !take_q();
            for (int32_t i = 0; i < n_pieces && !stop; ++i, ++np) {
                const int32_t tt = ms->piece[i].t, nt = ms->piece[i].j1 - ms->piece[i].j0;
                const int32_t slot = ms->piece[i].slot;
                float m = -INFINITY, l = 0.0f;  // running maximum (base 2); this thread's share of the sum
                uint32_t k = g - np - 1;  // key tiles so far
                for (int32_t j = 0; j < nt; ++j, ++g, ++k) {
                    ok = cx.wait(&ms->kv_full[g % kStages], (g / kStages) & 1, 30) &&
                         cx.wait(&ms->s_full, k & 1, 31);
                    tc::tc_fence_after();
                    const uint32_t valid = ms->valid[g % kStages][wg] >> (16 * hi);
                    float s[16];
                    // columns 64 wg on: groups of 8 keys, low and high dims in turn
                    if constexpr (Q4) {  // half of them at a time: 96 registers a thread
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            float c0[16], c1[16];
                            tc::tmem_ld16(lane_addr + kColS + 64 * wg + 16 * y, c0);
                            tc::tmem_ld16(lane_addr + kColS + 64 * wg + 32 + 16 * y, c1);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                const float own = hi ? c1[x + 8] : c0[x], give = hi ? c0[x + 8] : c1[x];
                                s[8 * y + x] = own + __shfl_xor_sync(0xffffffffu, give, 8);
                            }
                        }
                        tc::tc_fence_before();
                        tc::mbar_arrive(&ms->s_empty);
                    } else {
                        float c0[32], c1[32];
                        tc::tmem_ld32(lane_addr + kColS + 64 * wg, c0);
                        tc::tmem_ld32(lane_addr + kColS + 64 * wg + 32, c1);
                        tc::tmem_wait_ld();
                        tc::tc_fence_before();
                        tc::mbar_arrive(&ms->s_empty);
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const int c = 16 * (x >> 3) + (x & 7);  // low dims of key x of 16; high: + 8
                            const float own = hi ? c1[c + 8] : c0[c], give = hi ? c0[c + 8] : c1[c];
                            s[x] = own + __shfl_xor_sync(0xffffffffu, give, 8);
                        }
                    }
                    // Scores in base 2 above the running maximum, which the
                    // first tile sets (its largest weight is then exactly 1 in
                    // bf16) and later ones move only when a score exceeds it
                    // by more than kLazyMax, so that O^T is rarely rescaled;
                    // all softmax threads agree on it.
                    float v[16];
                    bool over = !ok || j == 0;
                    if (j > 0) {
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            v[x] = (valid >> x) & 1u ? fmaf(s[x], sc, -m) : -INFINITY;
                            over |= v[x] > kLazyMax;
                        }
                        over = any_of(over);
                    }
                    if (over) {
                        if (j > 0)
                            ok = ok && cx.wait(&ms->kv_empty[(g - 1) % kStages], ((g - 1) / kStages) & 1, 33);
                        float mt = -INFINITY;
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            v[x] = (valid >> x) & 1u ? s[x] * sc : -INFINITY;
                            mt = fmaxf(mt, v[x]);
                        }
                        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
                        float(*red)[64] = ms->red[k & 1];
                        if (!hi) red[wg][h] = mt;
                        if (!all_of(ok)) {
                            stop = true;
                            break;
                        }
                        mt = fmaxf(red[0][h], red[1][h]);
                        float al = 1.0f;
                        if (mt > m + kLazyMax) {  // always with the first keys: m is -inf
                            al = m == -INFINITY ? 1.0f : tc::ex2_approx(m - mt);
                            m = mt;
                        }
                        l *= al;
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            v[x] = m == -INFINITY ? v[x] : v[x] - m;  // no maximum yet: -inf or NaN
                        if (j > 0) {
                            if (wg == 0 && !hi) ms->fac[h] = al;
                            if (any_of(al != 1.0f)) {
                                tc::tc_fence_after();
                                const int h0 = 32 * wg;
#pragma unroll 1
                                for (int d = 0; d < 128 / kCols; ++d) {
                                    float o[kCols];
                                    const int x0 = h0 + kCols * d % 32;
                                    const uint32_t addr = lane_addr + kColO + 64 * (kCols * d / 32) + x0;
                                    tmem_ld<kCols>(addr, o);
                                    tc::tmem_wait_ld();
#pragma unroll
                                    for (int x = 0; x < kCols; ++x) o[x] *= ms->fac[x0 + x];
                                    tmem_st<kCols>(addr, o);
                                }
                                tc::tmem_wait_st();
                            }
                        }
                    }
                    // weights (bf16) -> 32 bytes of row h of P
                    unsigned char *prow = smem + kOffP + (k & 1) * 8192 + h * 128;
                    float sum = 0.0f;
#pragma unroll
                    for (int c8 = 0; c8 < 2; ++c8) {
                        uint32_t w4[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int x = 8 * c8 + 2 * y;
                            const float p0 = tc::ex2_approx(v[x]), p1 = tc::ex2_approx(v[x + 1]);
                            sum += p0 + p1;
                            const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
                            w4[y] = *reinterpret_cast<const uint32_t *>(&pb);
                        }
                        *reinterpret_cast<uint4 *>(prow + (((4 * wg + 2 * hi + c8) ^ (h & 7)) << 4)) =
                            make_uint4(w4[0], w4[1], w4[2], w4[3]);
                    }
                    l += sum;
                    tc::fence_proxy_async_smem();
                    tc::tc_fence_before();
                    tc::mbar_arrive(&ms->p_full[k & 1]);
                }
                if (stop) break;
                // the next piece's scores may start under this one's last O^T
                if (i + 1 < n_pieces && !take_q()) break;
                // ---- row sums, then O^T
                float(*red)[64] = ms->red[k & 1];  // no step of this token reads it any more
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                if (!hi) red[wg][h] = l;
                if (!all_of(ok)) {
                    stop = true;
                    break;
                }
                if (wg == 0 && !hi) {
                    l = red[0][h] + red[1][h];
                    float f = 1.0f;  // O^T times this
                    if (slot < 0) {
                        const float sk = a.sinks && h < a.H && ms->piece[i].k.seq >= 0
                                             ? __ldg(a.sinks + h) * kLog2e
                                             : -INFINITY;
                        const float M = fmaxf(m, sk);
                        const float w = m == -INFINITY ? 0.0f : tc::ex2_approx(m - M);
                        const float Z = fmaf(l, w, sk == -INFINITY ? 0.0f : tc::ex2_approx(sk - M));
                        f = Z == 0.0f ? 0.0f : w / Z;  // no key and no sink: 0; a NaN stays one
                        if (a.lse && h < a.H)
                            a.lse[(int64_t)tt * a.H + h] = (M + tc::lg2_approx(Z)) * kLn2;
                    } else {  // all 64: the join reads them by fours
                        ws.ml[slot * 64 + h] = make_float2(m, l);
                    }
                    ms->fac[h] = f;
                }
                ok = cx.wait(&ms->o_full, np & 1, 32);
                if (!all_of(ok)) {
                    stop = true;
                    break;
                }
                tc::tc_fence_after();
                // Lane of O^T slab d: dim 64 d + lane of the low (q4 < 2) or the
                // high half; heads 32 wg on
                const int h0 = 32 * wg, n_h = min(32, a.H - h0);
                const int dim = (q4 >> 1) * 256 + 32 * (q4 & 1) + lane;
                __nv_bfloat16 *outp = a.out + ((int64_t)tt * a.H + h0) * 512 + dim;
#pragma unroll 1
                for (int c = 0; c < 128 / kCols; ++c) {
                    const int d = kCols * c / 32, x0 = kCols * c % 32;
                    float o[kCols];
                    tmem_ld<kCols>(lane_addr + kColO + 64 * d + h0 + x0, o);
                    tc::tmem_wait_ld();
                    if (c + 1 == 128 / kCols) {  // O^T is read: the next token's may start
                        tc::tc_fence_before();
                        tc::mbar_arrive(&ms->o_empty);
                    }
                    if (slot >= 0) {
#pragma unroll
                        for (int x = 0; x < kCols; x += 4)
                            if (x0 + x < n_h)
                                *ws.sums(slot, (h0 + x0 + x) >> 2, dim + 64 * d) =
                                    make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
                    } else {
#pragma unroll
                        for (int x = 0; x < kCols; ++x)
                            if (x0 + x < n_h)
                                outp[(x0 + x) * 512 + 64 * d] = __float2bfloat16_rn(o[x] * ms->fac[h0 + x0 + x]);
                    }
                }
                tc::named_bar_sync(1, 256);  // fac and red are read
            }
        }
        __syncthreads();
        if (cx.aborted()) break;
    } while (ms->done < ms->run_e);  // written again behind a barrier of the next batch

    // ------------------------------------------------------------- teardown
    if (warp == 8 || warp == 9 || warp > kFindWarp) asm volatile("cp.async.wait_all;" ::: "memory");
    if (tid == 32 * kMmaWarp && issued) {  // no MMA outlives its tensor memory
        tc::mma_commit(&ms->drain);
        if (!tc::mbar_wait(&ms->drain, 0)) cx.fail(24);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

// Joins the tokens that several CTAs worked on. Block (x, y) takes token x
// (with more tokens than CTAs: the split token whose first tile CTA x held)
// and its items y, y + gridDim.y and so on: four heads and 256 ND / P dims, ND
// dims a thread, P groups of threads sharing the parts (ND = 1). Few blocks,
// three (ND = 1) or four an SM: they start only as the first kernel's CTAs
// leave (its registers fill the SM), and a grid of 32 blocks for each CTA, most
// without work, took 8 us to drain. The first parts' sums are on their way before their factors
// are known.
constexpr int kJoinThreads = 256;
constexpr int join_blocks(int nd) { return nd == 1 ? 3 : 4; }  // on an SM, by registers

template <int ND>
__global__ void __launch_bounds__(kJoinThreads, join_blocks(ND))
sparse_mla_paged_join_kernel(const __grid_constant__ MlaPagedArgs a, int32_t P) {
    __shared__ float w_s[4][kMaxGrid];
    __shared__ float inv_s[4];
    __shared__ float4 group_s[kJoinThreads];
    const Space ws(a.workspace, a.H);
    grid_dependency_wait();
    launch_dependents();
    const Join jn = ws.join[blockIdx.x];
    if (jn.first >= jn.last) return;  // one CTA had the whole token
    if (ND > 1) P = 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t parts = jn.last - jn.first + 1;
    const int32_t width = kJoinThreads / P, group = tid / width, dims = ND * width, slices = 512 / dims;
    // slot of part i: the first CTA's second slot, then the others' first ones
    auto slot = [&](int32_t i) { return 2 * (jn.first + i) + (i == 0 ? 1 : 0); };
    constexpr int kB = 8 / ND;
#pragma unroll 1
    for (int32_t item = blockIdx.y; item < ws.quads * slices; item += gridDim.y) {
        const int32_t quad = item / slices, dim = (item % slices) * dims + (tid - group * width);
        float4 v[kB][ND];
        auto fetch = [&](int32_t i0) {
#pragma unroll
            for (int i = 0; i < kB; ++i)
#pragma unroll
                for (int y = 0; y < ND; ++y)
                    if (i0 + P * i < parts) v[i][y] = *ws.sums(slot(i0 + P * i), quad, dim + y * kJoinThreads);
        };
        fetch(group);
        const int h = 4 * quad + warp;
        if (warp < 4) {  // one warp a head: the parts' factors
            const float sk = a.sinks && h < a.H ? __ldg(a.sinks + h) * kLog2e : -INFINITY;
            // a lane keeps its first part's pair; with more than 32 parts it reads the others twice
            const float2 first = lane < parts ? ws.ml[slot(lane) * 64 + h] : make_float2(-INFINITY, 0.0f);
            float M = fmaxf(sk, first.x);
            for (int32_t p = lane + 32; p < parts; p += 32) M = fmaxf(M, ws.ml[slot(p) * 64 + h].x);
            M = warp_max(M);
            float z = 0.0f;
            for (int32_t p = lane; p < parts; p += 32) {
                const float2 ml = p == lane ? first : ws.ml[slot(p) * 64 + h];
                const float f = ml.x == -INFINITY ? 0.0f : tc::ex2_approx(ml.x - M);
                w_s[warp][p] = f;
                z = fmaf(ml.y, f, z);
            }
            z = warp_sum(z) + (sk == -INFINITY ? 0.0f : tc::ex2_approx(sk - M));
            if (lane == 0) {
                inv_s[warp] = z == 0.0f ? 0.0f : 1.0f / z;  // a NaN stays one
                if (a.lse && h < a.H && item % slices == 0)
                    a.lse[(int64_t)jn.t * a.H + h] = (M + tc::lg2_approx(z)) * kLn2;
            }
        }
        __syncthreads();
        float o[ND][4] = {};
#pragma unroll 1
        for (int32_t i0 = group; i0 < parts; i0 += P * kB) {
            if (i0 != group) fetch(i0);
#pragma unroll
            for (int i = 0; i < kB; ++i) {
                const int32_t p = i0 + P * i;
                if (p < parts) {
                    const float f[4] = {w_s[0][p], w_s[1][p], w_s[2][p], w_s[3][p]};
#pragma unroll
                    for (int y = 0; y < ND; ++y) {
                        o[y][0] = fmaf(v[i][y].x, f[0], o[y][0]);
                        o[y][1] = fmaf(v[i][y].y, f[1], o[y][1]);
                        o[y][2] = fmaf(v[i][y].z, f[2], o[y][2]);
                        o[y][3] = fmaf(v[i][y].w, f[3], o[y][3]);
                    }
                }
            }
        }
        if (ND == 1 && P > 1) {
            group_s[tid] = make_float4(o[0][0], o[0][1], o[0][2], o[0][3]);
            __syncthreads();
            for (int q = 1; q < P && group == 0; ++q) {
                const float4 x = group_s[tid + q * width];
                o[0][0] += x.x;
                o[0][1] += x.y;
                o[0][2] += x.z;
                o[0][3] += x.w;
            }
        }
        if (group == 0)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (4 * quad + x < a.H) {
                    __nv_bfloat16 *out = a.out + ((int64_t)jn.t * a.H + 4 * quad + x) * 512 + dim;
                    const float r = inv_s[x];
#pragma unroll
                    for (int y = 0; y < ND; ++y) out[y * kJoinThreads] = __float2bfloat16_rn(o[y][x] * r);
                }
        __syncthreads();  // w_s, inv_s and group_s are read
    }
}

}  // namespace

size_t mla_paged_workspace_bytes(int32_t T, int32_t H) {
    if (T <= 0) return 0;
    return kMaxGrid * sizeof(Join) +
           (size_t)2 * kMaxGrid * (2 * 64 + (size_t)(H + 3) / 4 * 4 * 512) * sizeof(float);
}

namespace {

template <bool Q4>
cudaError_t launch(const MlaPagedArgs &a, cudaStream_t stream) {
    static PerContext pc;
    int sms, dev;
    bool first;
    unsigned long long ctx;
    cudaError_t e = enter_context(pc, &first, &ctx, &dev);
    if (e == cudaSuccess) e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    if (first) {
        e = cudaFuncSetAttribute(sparse_mla_paged_kernel<Q4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem_bytes<Q4>());
        if (e != cudaSuccess) return e;
        entered_context(pc, dev, ctx);
    }
    const int grid = min(sms, kMaxGrid);
    e = launch_early(sparse_mla_paged_kernel<Q4>, dim3(grid), dim3(Form<Q4>::kThreads), smem_bytes<Q4>(), stream, a);
    if (e != cudaSuccess) return e;
    // Small items while they fit at once: first the parts by four groups of
    // threads, then by two, then none, then two dims a thread.
    const int quads = (a.H + 3) / 4, gx = min(a.T, grid);
    for (int P = 4; P > 0; P >>= 1)
        if (2 * quads * gx * P <= join_blocks(1) * sms)
            return launch_early(sparse_mla_paged_join_kernel<1>, dim3(gx, 2 * quads * P), dim3(kJoinThreads), 0,
                                stream, a, (int32_t)P);
    return launch_early(sparse_mla_paged_join_kernel<2>, dim3(gx, max(1, min(quads, join_blocks(2) * sms / gx))),
                        dim3(kJoinThreads), 0, stream, a, 1);
}

}  // namespace

cudaError_t launch_sparse_mla_paged(MlaPagedArgs a, cudaStream_t stream) { return launch<false>(a, stream); }

cudaError_t launch_sparse_mla_paged_q4(MlaPagedArgs a, cudaStream_t stream) { return launch<true>(a, stream); }

}  // namespace csa
