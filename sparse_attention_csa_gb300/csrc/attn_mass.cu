// The attention weight that cached compressed rows received (sm_103a, tcgen05,
// cp.async):
//
//     out[b, j] = mass[b, j] + sum over the tokens t of sequence b that attend
//                 row j, and their heads h, of e^(scale q[t,h].k_j - lse[t,h])
//
// Two kernels. The first leaves the weight of every (token, key slot), heads
// summed, in the workspace; the second, one of two, adds a sequence's tokens up
// to a result that does not depend on the launch.
//
// Weights. The 128-slot tiles of all tokens are dealt to the CTAs in equal
// runs. A tile's rows are the MMA's M side, the heads its N side: S[j, h] =
// k_j . q_h over 512 dims, so that with one lane of tensor memory a row the sum
// over heads stays inside a thread, which takes e^(S - lse) as base-2
// exponentials. Rows of 4 bits come to shared memory as they are (48 KB a tile)
// and are turned into bf16 on the way to tensor memory, a thread a row: the
// MMA's A operand is read from there, so that shared memory carries 96 KB of
// rows and 64 KB of q a tile in place of 300 KB. Rows in bf16 are the operand
// in shared memory as they come.
//
// Sums. Weights are added in fixed point, two words of 64 bits, whose sums have
// no order (a row may be listed twice, and by several tokens): whole units, which
// leave room for every head of every token, and what they leave of a small
// weight. (In whole units alone, 2^-40 with 65535 tokens, weights below half of
// one were lost.) With lists a block has 2048 rows of one sequence in shared
// memory; without them 1024 in registers (six long rows, of units alone: 38.2 us;
// in shared memory as well 42.1).
//
// Bound by the latencies of both kernels' steps with few rows: one token of 512
// listed rows 11.6 us. 81 tokens' 41472 bf16 rows (42 MB) 23.5 us: at most three
// tiles a CTA, and the sums. Six long rows (84 MB in 4 bits) 38.3 us, 2.2 TB/s:
// 128 rows' MMAs take 67 clocks each, 2150 a tile, and the issuing thread some
// 600 a chunk besides; the turning of the rows takes as long beside it.
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "q4.cuh"
#include "tc_ptx.cuh"

namespace csa {

namespace {

// Key slots of token t: rows [0, vis) of sequence seq are visible, and its
// slots are the list's entries or these rows.
struct Slots {
    int32_t seq, vis, n;
};

__device__ __forceinline__ Slots token_slots(const MassArgs &a, int32_t t, bool report) {
    const int32_t pos = __ldg(a.q_pos + t);
    const int32_t b = paged_seq(a.q_seq, a.batch, t, pos);
    if (b < 0) {
        if (b == -2 && report) report_error(a.err, kErrCheck, kKerMass, 1);
        return {-1, 0, 0};
    }
    int32_t vis = (int32_t)(((uint32_t)pos + 1u) / (uint32_t)a.cmp_ratio);
    if (vis > a.max_rows) {
        if (report) report_error(a.err, kErrCheck, kKerMass, 2);
        vis = a.max_rows;
    }
    return {b, vis, a.idx ? (vis > 0 ? a.topk : 0) : vis};
}

// ------------------------------------------------------------------- weights
constexpr int kTile = 128;
constexpr int kPieces = 16;    // tokens of a run described in shared memory at a time
constexpr int kAcc = 2;        // tensor-memory accumulators of 64 columns
constexpr int kPresent = 8;    // tiles whose slots with a row are remembered
constexpr int kLoaders = 128;
// Rows of 4 bits enter the product without their power of two, which the sum's
// thread multiplies back: one multiplication a code in place of two. It is not
// taken below this, so that rotary dims beside vanishing others stay finite.
constexpr int kMinUp = -40;
constexpr float kLog2e = 1.4426950408889634f;

struct Piece {
    int32_t t, j0, j1;  // tiles [j0, j1) of token t
    Slots s;
};

// Q4 false: chunks of 128 rows x 128 dims in bf16 in shared memory. true: tiles
// of 4-bit rows there (raw), chunks of 256 dims in tensor memory. (A chunk costs
// the issuing thread some 600 clocks besides its MMAs, in a wait, a commit and
// their latencies: with chunks of 128 dims six long contexts took 47.7 us.)
template <bool Q4>
struct Form {
    static constexpr int kMmaWarp = Q4 ? 16 : 8;  // behind 4 epilogue, 4 loader and (Q4) 8 spread warps
    static constexpr int kThreads = 32 * (kMmaWarp + 1);
    static constexpr int kRaw = Q4 ? 2 : 0;
    static constexpr int kPerTile = Q4 ? 2 : 4;   // chunks
    static constexpr int kChunks = 3;             // at a time, of 128 columns or 32 KB
    static constexpr int kMmas = 32 / kPerTile;   // of a chunk, 16 dims each
    static constexpr uint32_t kQ = 64 * 512 * 2;
    static constexpr uint32_t kOffQ = 0;          // two tokens' heads
    static constexpr uint32_t kOffRows = 2 * kQ;
    static constexpr uint32_t kRawTile = kTile * q4::kRow;
    static constexpr uint32_t kChunkBytes = kTile * 256;
    static constexpr uint32_t kOffMisc = kOffRows + (Q4 ? kRaw * kRawTile : kChunks * kChunkBytes);
    static constexpr uint32_t kColChunk = 64 * kAcc;
    static constexpr uint32_t kCols = Q4 ? 512 : 128;
    static_assert(!Q4 || kColChunk + 128 * kChunks <= kCols, "tensor memory");
    static_assert((int64_t)kThreads * (kMaxKeys / kTile) <= INT32_MAX, "a scan's sum");
};

template <bool Q4>
struct Misc {
    using F = Form<Q4>;
    uint64_t q_full[2], q_empty[2];
    uint64_t raw_full[2], raw_empty[2];
    uint64_t chunk_full[F::kChunks], chunk_empty[F::kChunks];
    uint64_t acc_full[kAcc], acc_empty[kAcc];
    uint64_t present_full[kPresent];  // which slots have a row (loaders) and their powers of two (spread warps)
    uint64_t drain;
    int64_t run_base, done;
    int32_t run_t, n_pieces;
    uint32_t tmem_base;
    int32_t abort;
    int32_t scan[F::kThreads / 32 + 1];
    uint32_t present[kPresent][4];
    int8_t up[kPresent][kTile];  // powers of two taken out of the rows (4 bits)
    Piece piece[kPieces];
    alignas(16) float lse2[4][64];  // each epilogue warp's own
};

template <bool Q4>
constexpr size_t smem_bytes() {
    return Form<Q4>::kOffMisc + sizeof(Misc<Q4>);
}
static_assert(smem_bytes<false>() <= 232448 && smem_bytes<true>() <= 232448, "shared memory budget");

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

__device__ __forceinline__ void tmem_st_words(uint32_t taddr, const uint4 (&v)[4]) {
    float f[16];  // the bits as they are
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[4 * i] = __uint_as_float(v[i].x);
        f[4 * i + 1] = __uint_as_float(v[i].y);
        f[4 * i + 2] = __uint_as_float(v[i].z);
        f[4 * i + 3] = __uint_as_float(v[i].w);
    }
    tc::tmem_st16(taddr, f);
}

template <bool Q4>
__global__ void __launch_bounds__(Form<Q4>::kThreads, 1)
attn_weight_kernel(const __grid_constant__ MassArgs a) {
    using F = Form<Q4>;
    constexpr int kThreads = F::kThreads, kMmaWarp = F::kMmaWarp, kChunks = F::kChunks;
    constexpr int kRaw = Q4 ? F::kRaw : 1;
    extern __shared__ __align__(1024) unsigned char smem[];  // swizzled tiles: lines of 8 x 128 bytes
    Misc<Q4> *ms = reinterpret_cast<Misc<Q4> *>(smem + F::kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PipeWaits<Misc<Q4>, kKerMass> cx{ms, a.err, a.wait_ns};
    const int32_t c = blockIdx.x;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&ms->q_full[i], kLoaders);
            tc::mbar_init(&ms->q_empty[i], 1);
            tc::mbar_init(&ms->raw_full[i], kLoaders);
            tc::mbar_init(&ms->raw_empty[i], 8);
        }
        for (int i = 0; i < kChunks; ++i) {
            tc::mbar_init(&ms->chunk_full[i], Q4 ? 4 : kLoaders);
            tc::mbar_init(&ms->chunk_empty[i], 1);
        }
        for (int i = 0; i < kAcc; ++i) {
            tc::mbar_init(&ms->acc_full[i], 1);
            tc::mbar_init(&ms->acc_empty[i], 128);
        }
        for (int i = 0; i < kPresent; ++i) tc::mbar_init(&ms->present_full[i], Q4 ? 8 : 4);
        tc::mbar_init(&ms->drain, 1);
        ms->abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&ms->tmem_base, F::kCols);
        tc::tmem_relinquish();
    }
    // heads past H: zero rows of both q buffers, never written again
    for (int i = tid; i < 2 * (64 - a.H) * 64; i += kThreads) {
        const int buf = i / ((64 - a.H) * 64), r = i - buf * (64 - a.H) * 64, h = a.H + (r >> 6), u = r & 63;
        *reinterpret_cast<uint4 *>(smem + F::kOffQ + buf * F::kQ + (u >> 3) * 8192 + h * 128 + (u & 7) * 16) =
            make_uint4(0, 0, 0, 0);
    }
    // everything above is local: wait for the kernels before this one
    grid_dependency_wait();
    launch_dependents();
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();

    // ------------------------------------------------ this CTA's run of tiles
    const bool one_scan = a.T <= kThreads;
    Slots sl = {-1, 0, 0};
    int32_t nt = 0, total = 0;
    int64_t N = 0, b = 0;  // tiles in all, and before the thread's token
    for (int32_t t0 = 0; t0 < a.T; t0 += kThreads) {
        const int32_t t = t0 + tid;
        sl = {-1, 0, 0};
        if (t < a.T) sl = token_slots(a, t, c == 0);
        nt = (sl.n + kTile - 1) / kTile;
        b = block_exclusive_scan<kThreads>(nt, ms->scan, &total);
        N += total;
    }
    tc::tc_fence_after();
    const uint32_t tmem = ms->tmem_base;
    const int64_t per = div64(N + gridDim.x - 1, gridDim.x);
    const int64_t s = min(c * per, N), e = min(s + per, N);
    if (s == e) {  // no run left for this CTA
        __syncthreads();
        if (warp == kMmaWarp) tc::tmem_dealloc(tmem, F::kCols);
        return;
    }
    if (one_scan) {
        if (b <= s && s < b + nt) ms->run_t = tid;
    } else {  // the token holding tile s
        int64_t base = 0;
        for (int32_t t0 = 0; t0 < a.T && base <= s; t0 += kThreads) {
            const int32_t t = t0 + tid;
            const int32_t k = t < a.T ? (token_slots(a, t, false).n + kTile - 1) / kTile : 0;
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
            sl = {-1, 0, 0};
            if (tid < kPieces && t < a.T) sl = token_slots(a, t, false);
            nt = (sl.n + kTile - 1) / kTile;
            b = base + block_exclusive_scan<kThreads>(nt, ms->scan, &total);
        }
        if (x >= 0 && x < kPieces && t < a.T && b < e) {  // a token without tiles has an empty piece
            ms->piece[x] = {t, (int32_t)max(s - b, (int64_t)0), (int32_t)min(e - b, (int64_t)nt), sl};
            if (x == kPieces - 1 || t + 1 == a.T || b + nt >= e) {
                ms->n_pieces = x + 1;
                ms->done = min(e, b + nt);
            }
        }
        __syncthreads();
        if (tid == 0) {
            ms->run_t = t_first + kPieces;
            if (!one_scan) ms->run_base += total;
        }
        done = ms->done;
        const int32_t n_pieces = ms->n_pieces;

        if (warp == kMmaWarp) {
            // ===================================================== MMA warp
            if (lane == 0) {
                constexpr uint32_t id = tc::idesc_bf16(128, 64, false, false);
                const uint64_t da = tc::smem_desc(tc::smem_u32(smem + F::kOffRows), 16, 1024);
                const uint64_t db = tc::smem_desc(tc::smem_u32(smem + F::kOffQ), 16, 1024);
                bool ok = true;
                for (int32_t i = 0; i < n_pieces && ok; ++i) {
                    const int32_t j0 = ms->piece[i].j0, j1 = ms->piece[i].j1;
                    if (j0 >= j1) continue;
                    ok = cx.wait(&ms->q_full[np & 1], (np >> 1) & 1, 20);
                    tc::fence_proxy_async_smem();  // cp.async wrote through the generic proxy
                    for (int32_t j = j0; j < j1 && ok; ++j, ++g) {
                        const uint32_t acc = g % kAcc;
                        ok = cx.wait(&ms->acc_empty[acc], ((g / kAcc) & 1) ^ 1, 22);
#pragma unroll 1
                        for (uint32_t ch = 0; ch < F::kPerTile && ok; ++ch) {
                            const uint32_t cc = F::kPerTile * g + ch, st = cc % kChunks;
                            ok = tc::mbar_test(&ms->chunk_full[st], (cc / kChunks) & 1) ||
                                 cx.wait(&ms->chunk_full[st], (cc / kChunks) & 1, 21);
                            if (!ok) break;
                            if constexpr (!Q4) tc::fence_proxy_async_smem();
                            tc::tc_fence_after();
                            const uint64_t bq = tc::desc_add(db, (np & 1) * F::kQ + ch * (F::kMmas * 2048));
#pragma unroll
                            for (int kk = 0; kk < F::kMmas; ++kk) {
                                const uint64_t b = tc::desc_add(bq, (kk >> 2) * 8192 + (kk & 3) * 32);
                                if constexpr (Q4)
                                    mma_bf16_ta(tmem + 64 * acc, tmem + F::kColChunk + 128 * st + 8 * kk, b, id,
                                                (ch | kk) != 0);
                                else
                                    tc::mma_bf16(tmem + 64 * acc,
                                                 tc::desc_add(da, st * F::kChunkBytes + (kk >> 2) * 16384 +
                                                                      (kk & 3) * 32),
                                                 b, id, (ch | kk) != 0);
                            }
                            issued = true;
                            tc::mma_commit(&ms->chunk_empty[st]);
                        }
                        if (ok) tc::mma_commit(&ms->acc_full[acc]);
                    }
                    if (ok) tc::mma_commit(&ms->q_empty[np & 1]);
                    ++np;
                }
            }
            __syncwarp();
        } else if (warp >= 8) {
            // ================================================= spread warps
            // Four warps have the 128 rows, a thread one; two sets of them take
            // turns with the chunks. A row's 14 pieces of 32 codes lie in 16-byte
            // places permuted within its lines, so that 8 lanes meet no bank twice.
            if constexpr (Q4) {
                const int quarter = warp & 3, set = (warp - 8) >> 2, sw = (lane & 7) << 4;
                const uint32_t col = tmem + ((uint32_t)(32 * quarter) << 16) + F::kColChunk;
                bool ok = true;
                for (int32_t i = 0; i < n_pieces && ok; ++i) {
                    const int32_t j0 = ms->piece[i].j0, j1 = ms->piece[i].j1;
                    for (int32_t j = j0; j < j1; ++j, ++g) {
                        const uint32_t rs = g % kRaw;
                        ok = __all_sync(0xffffffffu, cx.wait(&ms->raw_full[rs], (g / kRaw) & 1, 50));
                        if (!ok) break;
                        const unsigned char *row =
                            smem + F::kOffRows + rs * F::kRawTile + (32 * quarter + lane) * q4::kRow;
                        const int ex = (int)row[q4::kExp ^ sw] - 127;
                        // codes times this times their scale are the row over 2^(up + 8)
                        const float unit = q4::pow2(118 + min(ex - kMinUp, 0));
                        const __nv_bfloat162 down = __float2bfloat162_rn(q4::pow2(-max(ex, kMinUp) - 8));
                        if (set == 0) {
                            ms->up[g % kPresent][32 * quarter + lane] = (int8_t)max(ex, kMinUp);
                            __syncwarp();
                            if (lane == 0) tc::mbar_arrive(&ms->present_full[g % kPresent]);
                        }
                        const uint32_t cc = 2 * g + set, st = cc % kChunks;
                        ok = __all_sync(0xffffffffu,
                                        cx.wait(&ms->chunk_empty[st], ((cc / kChunks) & 1) ^ 1, 51));
                        if (!ok) break;
                        tc::tc_fence_after();
                        // four groups' scales at a time, of two pieces of 32 dims
#pragma unroll 1
                        for (int p = 0; p < 4; ++p) {
                            const int piece = 8 * set + 2 * p;
                            const uint32_t at = col + 128 * st + 32 * p;
                            if (piece < 14) {
                                const uint32_t four = *reinterpret_cast<const uint32_t *>(
                                    row + ((q4::kScales + 2 * piece) ^ sw));
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    const uint4 w = *reinterpret_cast<const uint4 *>(row + ((16 * (piece + x)) ^ sw));
                                    const float2 f = q4::scales2((uint16_t)(four >> (16 * x)));
                                    const __nv_bfloat162 s0 = q4::scale_pair(f.x, unit);
                                    const __nv_bfloat162 s1 = q4::scale_pair(f.y, unit);
                                    const uint4 v[4] = {q4::times(q4::eight_small(w.x), s0),
                                                        q4::times(q4::eight_small(w.y), s0),
                                                        q4::times(q4::eight_small(w.z), s1),
                                                        q4::times(q4::eight_small(w.w), s1)};
                                    tmem_st_words(at + 16 * x, v);
                                }
                            } else {
#pragma unroll 1
                                for (int x = 0; x < 2; ++x) {
                                    uint4 v[4];
#pragma unroll
                                    for (int y = 0; y < 4; ++y)
                                        v[y] = q4::times(*reinterpret_cast<const uint4 *>(
                                                             row + ((q4::kTail + 64 * x + 16 * y) ^ sw)),
                                                         down);
                                    tmem_st_words(at + 16 * x, v);
                                }
                            }
                        }
                        tc::tmem_wait_st();
                        tc::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            tc::mbar_arrive(&ms->chunk_full[st]);
                            tc::mbar_arrive(&ms->raw_empty[rs]);
                        }
                    }
                }
            }
        } else if (warp >= 4) {
            // ================================================= loader warps
            // Warp w: slots 32 w .. 32 w + 31 of every tile, one a lane. Finding a
            // row takes two dependent loads (the list's entry, the page); they run
            // two tiles and one tile ahead.
            const int w = warp - 4, li = tid - 128;
            bool ok = true;
            for (int32_t i = 0; i < n_pieces && ok; ++i) {
                const Piece p = ms->piece[i];
                if (p.j0 >= p.j1) continue;
                auto row_at = [&](int32_t j) -> int32_t {
                    const int64_t x = (int64_t)j * kTile + 32 * w + lane;
                    if (j >= p.j1 || x >= p.s.n) return -1;
                    const int32_t r = a.idx ? __ldg(a.idx + (int64_t)p.t * a.topk + x) : (int32_t)x;
                    return r < p.s.vis ? r : -1;
                };
                auto page_of = [&](int32_t r, int32_t *in) -> int32_t {
                    *in = -1;
                    if (r < 0) return -1;
                    const uint32_t pg = (uint32_t)r / (uint32_t)a.cmp.page_size;  // in the table: r < max_rows
                    *in = r - (int32_t)pg * a.cmp.page_size;
                    return __ldg(a.cmp.pages + (int64_t)p.s.seq * a.cmp.max_pages + pg);
                };
                int32_t in, row_next = row_at(p.j0 + 1);
                int32_t page = page_of(row_at(p.j0), &in);
                ok = __all_sync(0xffffffffu, cx.wait(&ms->q_empty[np & 1], ((np >> 1) & 1) ^ 1, 40));
                if (!ok) break;
                {
                    const __nv_bfloat16 *q = a.q + (int64_t)p.t * a.H * 512;
                    const uint32_t dst = tc::smem_u32(smem + F::kOffQ) + (np & 1) * F::kQ;
#pragma unroll 4
                    for (int u = li; u < a.H * 64; u += kLoaders) {
                        const int h = u >> 6, y = u & 63;
                        cp_async16(dst + (y >> 3) * 8192 + h * 128 + (((y ^ h) & 7) << 4), q + (int64_t)u * 8, 16);
                    }
                }
                cp_async_arrive(&ms->q_full[np & 1]);
                ++np;
                for (int32_t j = p.j0; j < p.j1; ++j, ++g) {
                    const unsigned char *mine = nullptr;
                    if (in >= 0) {
                        if ((uint32_t)page < (uint32_t)a.cmp.num_pages)
                            mine = reinterpret_cast<const unsigned char *>(a.cmp.base) +
                                   ((int64_t)page * a.cmp.page_size + in) * (Q4 ? q4::kRow : 1024);
                        else if (page != CSA_PAGE_EVICTED)
                            report_error(a.err, kErrCheck, kKerMass, 3);
                    }
                    const uint32_t m = __ballot_sync(0xffffffffu, mine != nullptr);
                    page = page_of(row_next, &in);
                    row_next = row_at(j + 2);
                    if constexpr (Q4) {
                        const uint32_t rs = g % kRaw;
                        ok = __all_sync(0xffffffffu, cx.wait(&ms->raw_empty[rs], ((g / kRaw) & 1) ^ 1, 41));
                        if (!ok) break;
                        // four rows of 384 bytes are three instructions
                        const uint32_t raw =
                            tc::smem_u32(smem + F::kOffRows) + rs * F::kRawTile + 32 * w * q4::kRow;
#pragma unroll 1
                        for (int x = 0; x < 3; ++x) {
                            const int sub = (32 * x + lane) / 24, piece = (32 * x + lane) % 24;
#pragma unroll
                            for (int r = 0; r < 32; r += 4) {
                                const unsigned char *src = reinterpret_cast<const unsigned char *>(
                                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), r + sub));
                                const uint32_t bytes = src ? 16u : 0u;  // no row: zeros
                                if (!src) src = reinterpret_cast<const unsigned char *>(a.q);
                                cp_async16(raw + (r + sub) * q4::kRow + (16 * piece ^ (((r + sub) & 7) << 4)),
                                           src + 16 * piece, bytes);
                            }
                        }
                        cp_async_arrive(&ms->raw_full[rs]);
                    } else {
#pragma unroll 1
                        for (uint32_t ch = 0; ch < 4; ++ch) {
                            const uint32_t cc = 4 * g + ch, st = cc % kChunks;
                            ok = __all_sync(0xffffffffu,
                                            cx.wait(&ms->chunk_empty[st], ((cc / kChunks) & 1) ^ 1, 42));
                            if (!ok) break;
                            // two rows' 256 bytes an instruction
                            const int y = lane & 15, sub = lane >> 4;
                            const uint32_t base_s = tc::smem_u32(smem + F::kOffRows) + st * F::kChunkBytes +
                                                    (y >> 3) * 16384 + 32 * w * 128;
#pragma unroll
                            for (int r = 0; r < 32; r += 2) {
                                const unsigned char *src = reinterpret_cast<const unsigned char *>(
                                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), r + sub));
                                const uint32_t bytes = src ? 16u : 0u;
                                if (!src) src = reinterpret_cast<const unsigned char *>(a.q);
                                cp_async16(base_s + (r + sub) * 128 + (((y ^ (r + sub)) & 7) << 4),
                                           src + 256 * ch + 16 * y, bytes);
                            }
                            cp_async_arrive(&ms->chunk_full[st]);
                        }
                        if (!ok) break;
                    }
                    if (lane == 0) {
                        // read long before tile g + kPresent: at most four tiles lie
                        // between these warps and the epilogue
                        ms->present[g % kPresent][w] = m;
                        tc::mbar_arrive(&ms->present_full[g % kPresent]);
                    }
                }
            }
        } else {
            // =============================================== epilogue warps
            const uint32_t lane_addr = tmem + ((uint32_t)(32 * warp) << 16);
            const float sc = a.softmax_scale * kLog2e;
            bool ok = true;
            for (int32_t i = 0; i < n_pieces && ok; ++i) {
                const Piece p = ms->piece[i];
                if (p.j0 >= p.j1) continue;
                float *lse2 = ms->lse2[warp];
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 2; ++x) {  // +inf: a head that counts nothing
                    const int h = 32 * x + lane;
                    const float l = h < a.H ? __ldg(a.lse + (int64_t)p.t * a.H + h) : -INFINITY;
                    lse2[h] = l == -INFINITY ? INFINITY : l * kLog2e;
                }
                __syncwarp();
                float *out = a.weights + (int64_t)p.t * a.slot_pad;
                for (int32_t j = p.j0; j < p.j1; ++j, ++g) {
                    const uint32_t acc = g % kAcc;
                    ok = __all_sync(0xffffffffu,
                                    cx.wait(&ms->present_full[g % kPresent], (g / kPresent) & 1, 31) &&
                                        cx.wait(&ms->acc_full[acc], (g / kAcc) & 1, 32));
                    if (!ok) break;
                    tc::tc_fence_after();
                    const bool there = (ms->present[g % kPresent][warp] >> lane) & 1u;
                    const float scr = Q4 ? sc * q4::pow2(ms->up[g % kPresent][32 * warp + lane] + 8) : sc;
                    float sum[2] = {0.0f, 0.0f};
#pragma unroll 1
                    for (int h = 0; h < 64; h += 16) {
                        float v[16];
                        tc::tmem_ld16(lane_addr + 64 * acc + h, v);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int y = 0; y < 16; y += 4) {
                            const float4 l = *reinterpret_cast<const float4 *>(lse2 + h + y);
                            sum[0] += tc::ex2_approx(fmaf(v[y], scr, -l.x));
                            sum[1] += tc::ex2_approx(fmaf(v[y + 1], scr, -l.y));
                            sum[0] += tc::ex2_approx(fmaf(v[y + 2], scr, -l.z));
                            sum[1] += tc::ex2_approx(fmaf(v[y + 3], scr, -l.w));
                        }
                    }
                    tc::tc_fence_before();
                    tc::mbar_arrive(&ms->acc_empty[acc]);
                    // NaN counts as 0; more than one a head only an lse that is not the attention's can give
                    const float all = sum[0] + sum[1], most = (float)a.H;
                    out[(int64_t)j * kTile + 32 * warp + lane] =
                        there && all <= most ? all : there && all > most ? most : 0.0f;
                }
            }
        }
        __syncthreads();
        if (cx.aborted()) break;
    }

    // ------------------------------------------------------------- teardown
    if (warp >= 4 && warp < 8) asm volatile("cp.async.wait_all;" ::: "memory");
    if (tid == 32 * kMmaWarp && issued) {  // no MMA outlives its tensor memory
        tc::mma_commit(&ms->drain);
        if (!tc::mbar_wait(&ms->drain, 0)) cx.fail(24);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, F::kCols);
}

// ---------------------------------------------------------------------- sums
// One block on an SM is asked for: left to itself the compiler keeps to 32
// registers and spills (one token, of units alone: 14.0 us in place of 12.4).
constexpr int kSumThreads = 256;
constexpr int kTokens = 512;  // of the sequence, known at a time

// Weights in fixed point: whole units of 2^-lg_unit, and what they leave in parts
// of 2^-lg_part of a unit. Shifts of the mantissa, exact but for the rounding
// below one part. (Conversions to 64 bits in their place, of which the SM does
// few: 2048 tokens' weights of all rows 1560 us where shifts took 914.)
struct Fixed {
    unsigned long long units, parts;
};
__device__ __forceinline__ Fixed fixed_point(const MassArgs &a, float x) {
    const uint32_t bits = __float_as_uint(x);  // not negative
    if (bits < 0x800000u) return {0, 0};       // below any part: lg_unit + lg_part <= 119
    const uint32_t m = (bits & 0x7fffffu) | 0x800000u;
    const int e = (int)(bits >> 23) - 150 + a.lg_unit;  // m 2^e units
    if (e >= 0) return {(unsigned long long)m << e, 0};
    const int below = min(-e, 24), up = a.lg_part + e;
    const uint32_t left = m & ((1u << below) - 1u);
    return {m >> below, up >= 0    ? (unsigned long long)left << up
                        : up > -25 ? (unsigned long long)((left + (1u << (-up - 1))) >> -up)
                                   : 0};
}
__device__ __forceinline__ float weight_of(const MassArgs &a, const Fixed &f) {
    return fmaf(__ull2float_rn(f.parts), q4::pow2(-a.lg_unit - a.lg_part),
                __ull2float_rn(f.units) * q4::pow2(-a.lg_unit));
}

// Without lists: a thread's four rows keep their sums in registers.
constexpr int kAllMine = 4;
constexpr int kAllRows = kAllMine * kSumThreads;

__global__ void __launch_bounds__(kSumThreads, 1) attn_mass_all_kernel(const __grid_constant__ MassArgs a) {
    __shared__ int32_t token[kTokens], slots[kTokens];
    __shared__ int32_t n_tokens;
    const int tid = threadIdx.x;
    const int32_t b = blockIdx.y, r0 = blockIdx.x * kAllRows, n = min(kAllRows, a.max_rows - r0);
    const int64_t row = (int64_t)b * a.max_rows + r0;
    const bool in_place = a.out == a.mass;
    if (tid == 0) n_tokens = 0;
    __syncthreads();
    grid_dependency_wait();
    launch_dependents();
    // what the sums are added to is on its way while they are formed (in place
    // only rows with weight are touched)
    float old[kAllMine];
    Fixed sum[kAllMine] = {};
#pragma unroll
    for (int i = 0; i < kAllMine; ++i)
        old[i] = !in_place && a.mass && tid + i * kSumThreads < n ? __ldg(a.mass + row + tid + i * kSumThreads) : 0.0f;
    for (int32_t t0 = 0; t0 < a.T; t0 += kTokens) {
        // the sequence's tokens, in any order: sums have none
#pragma unroll
        for (int x = 0; x < kTokens; x += kSumThreads) {
            const int32_t t = t0 + x + tid;
            if (t < a.T) {
                const Slots s = token_slots(a, t, false);
                if (s.seq == b && s.n > r0) {
                    const int32_t at = atomicAdd(&n_tokens, 1);
                    token[at] = t;
                    slots[at] = s.n;
                }
            }
        }
        __syncthreads();
        const int32_t nt = n_tokens;
        __syncthreads();
        if (tid == 0) n_tokens = 0;
        // the next token's weights are on their way while one's are added (2048
        // tokens of one sequence 717 us; one token after the other 914)
        float next[kAllMine];
        auto fetch = [&](int32_t k) {
            const float *w = a.weights + (int64_t)token[k] * a.slot_pad + r0;
            const int32_t m = min(n, slots[k] - r0);
#pragma unroll
            for (int i = 0; i < kAllMine; ++i) next[i] = tid + i * kSumThreads < m ? w[tid + i * kSumThreads] : 0.0f;
        };
        if (nt > 0) fetch(0);
#pragma unroll 1
        for (int32_t k = 0; k < nt; ++k) {
            float x[kAllMine];
#pragma unroll
            for (int i = 0; i < kAllMine; ++i) x[i] = next[i];
            if (k + 1 < nt) fetch(k + 1);
#pragma unroll
            for (int i = 0; i < kAllMine; ++i) {
                const Fixed f = fixed_point(a, x[i]);
                sum[i].units += f.units;
                sum[i].parts += f.parts;
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kAllMine; ++i) {
        const int r = tid + i * kSumThreads;
        if (r >= n) break;
        if (sum[i].units | sum[i].parts)
            a.out[row + r] = (in_place ? a.out[row + r] : old[i]) + weight_of(a, sum[i]);
        else if (!in_place) a.out[row + r] = old[i];
    }
}

// With lists: a block's rows keep their sums in shared memory.
constexpr int kListRows = 2048;
constexpr int kListMine = kListRows / kSumThreads;  // rows a thread finishes

__global__ void __launch_bounds__(kSumThreads, 1) attn_mass_list_kernel(const __grid_constant__ MassArgs a) {
    __shared__ unsigned long long units[kListRows], parts[kListRows];
    __shared__ int32_t token[kTokens], slots[kTokens], seen[kTokens];
    __shared__ int32_t n_tokens;
    const int tid = threadIdx.x;
    const int32_t b = blockIdx.y, r0 = blockIdx.x * kListRows, n = min(kListRows, a.max_rows - r0);
    const int64_t row = (int64_t)b * a.max_rows + r0;
    const bool in_place = a.out == a.mass;
    for (int i = tid; i < n; i += kSumThreads) units[i] = parts[i] = 0;
    if (tid == 0) n_tokens = 0;
    __syncthreads();
    grid_dependency_wait();
    launch_dependents();
    // what the sums are added to is on its way while they are formed (in place
    // only rows with weight are touched)
    float old[kListMine];
#pragma unroll
    for (int i = 0; i < kListMine; ++i)
        old[i] = !in_place && a.mass && tid + i * kSumThreads < n ? __ldg(a.mass + row + tid + i * kSumThreads) : 0.0f;
    for (int32_t t0 = 0; t0 < a.T; t0 += kTokens) {
        // the sequence's tokens, in any order: sums have none
#pragma unroll
        for (int x = 0; x < kTokens; x += kSumThreads) {
            const int32_t t = t0 + x + tid;
            if (t < a.T) {
                const Slots s = token_slots(a, t, false);
                if (s.seq == b && s.n > 0) {
                    const int32_t at = atomicAdd(&n_tokens, 1);
                    token[at] = t;
                    slots[at] = s.n;
                    seen[at] = s.vis;
                }
            }
        }
        __syncthreads();
        const int32_t nt = n_tokens;
        __syncthreads();
        if (tid == 0) n_tokens = 0;
        for (int32_t k = 0; k < nt; ++k) {
            const float *w = a.weights + (int64_t)token[k] * a.slot_pad;
            const int32_t *list = a.idx + (int64_t)token[k] * a.topk;
            const int32_t end = min(r0 + n, seen[k]);
            // two entries at a time, added one after the other: the code of an
            // addition four times over took 0.6 us more for 81 tokens
            for (int32_t i = tid; i < slots[k]; i += 2 * kSumThreads) {
                const bool two = i + kSumThreads < slots[k];
                int32_t r = __ldg(list + i), r_next = two ? __ldg(list + i + kSumThreads) : -1;
                float x = w[i], x_next = two ? w[i + kSumThreads] : 0.0f;
#pragma unroll 1
                for (int y = 0; y < 2; ++y, r = r_next, x = x_next) {
                    if (r < r0 || r >= end || x == 0.0f) continue;
                    const Fixed f = fixed_point(a, x);
                    if (f.units) atomicAdd(&units[r - r0], f.units);
                    if (f.parts) atomicAdd(&parts[r - r0], f.parts);
                }
            }
        }
        __syncthreads();
    }
    Fixed sum[kListMine];
#pragma unroll
    for (int i = 0; i < kListMine; ++i) {
        const int r = tid + i * kSumThreads;
        sum[i] = r < n ? Fixed{units[r], parts[r]} : Fixed{0, 0};
        if (in_place && (sum[i].units | sum[i].parts)) old[i] = a.out[row + r];
    }
#pragma unroll
    for (int i = 0; i < kListMine; ++i) {
        const int r = tid + i * kSumThreads;
        if (r >= n) break;
        if (sum[i].units | sum[i].parts) a.out[row + r] = old[i] + weight_of(a, sum[i]);
        else if (!in_place) a.out[row + r] = old[i];
    }
}

template <bool Q4>
cudaError_t launch_weights(const MassArgs &a, cudaStream_t stream) {
    static PerContext pc;
    int sms, dev;
    bool first;
    unsigned long long ctx;
    cudaError_t e = enter_context(pc, &first, &ctx, &dev);
    if (e == cudaSuccess) e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    if (first) {
        e = cudaFuncSetAttribute(attn_weight_kernel<Q4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem_bytes<Q4>());
        if (e != cudaSuccess) return e;
        entered_context(pc, dev, ctx);
    }
    return launch_early(attn_weight_kernel<Q4>, dim3(sms), dim3(Form<Q4>::kThreads), smem_bytes<Q4>(), stream, a);
}

}  // namespace

int64_t mass_slot_pad(int64_t slots) { return (slots + kTile - 1) / kTile * kTile; }

size_t mass_workspace_bytes(int32_t T, int64_t slots) {
    return T > 0 ? (size_t)T * (size_t)mass_slot_pad(slots) * 4 : 0;
}

cudaError_t launch_attn_mass(MassArgs a, cudaStream_t stream) {
    if (a.T > 0) {
        const cudaError_t e = a.q4 ? launch_weights<true>(a, stream) : launch_weights<false>(a, stream);
        if (e != cudaSuccess) return e;
    }
    const auto sums = a.idx ? attn_mass_list_kernel : attn_mass_all_kernel;
    const int rows = a.idx ? kListRows : kAllRows;
    return launch_early(sums, dim3((unsigned)(((int64_t)a.max_rows + rows - 1) / rows), a.batch), dim3(kSumThreads), 0,
                        stream, a);
}

}  // namespace csa
