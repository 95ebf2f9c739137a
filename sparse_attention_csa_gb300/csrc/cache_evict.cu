// Pages of cached rows to give back, by the attention weight their rows
// received (sm_103a).
//
//     weight of page p = sum of mass[b, r] over its rows r in use
// Of the pages a sequence holds, those with rows that are to stay (the first,
// the last, and a page with room for the next ones) stay; of the others the
// heaviest stay while the budget lasts, the lower page among equals. The rest
// are marked in the table and listed.
//
// One block a sequence. Groups of lanes sum a page each, as a 32-bit sum and
// the sum of its rounding errors (each found exactly by Knuth's two-sum), so
// that the order of the rows does not decide between two pages: 64-bit
// additions, of which the SM does two a clock, made it 44 us for 512 pages and
// 83 us for 64 sequences. The border between staying and going is found by
// halving the interval of the sums' keys and counting, which ends as soon as a
// value parts them right: some 12 counts for 512 pages, 64 at most (equal sums).
#include "common.cuh"
#include "internal.h"
#include "paged.h"

namespace csa {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// A sum and what its roundings left out.
struct Sum {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float x) {
        const float s = hi + x, b = s - hi;
        lo += (hi - (s - b)) + (x - b);
        hi = s;
    }
    // Order-preserving map of hi + lo to uint64, above 0; NaN above all. The
    // first word is the sum rounded to 32 bits, the second what is left of it.
    __device__ __forceinline__ uint64_t key() const {
        if (hi != hi) return ~0ull;
        float h = hi, l = 0.0f;
        if (fabsf(hi) <= 3.402823466e38f) {
            h = hi + lo;
            l = lo - (h - hi);
        }
        return (uint64_t)float_key(h) << 32 | float_key(l);
    }
};

__global__ void __launch_bounds__(kThreads) cache_evict_kernel(const __grid_constant__ EvictArgs a) {
    extern __shared__ uint64_t key[];  // of each page: 0, stays or is not held
    __shared__ int32_t scan[kWarps + 1];
    __shared__ int32_t count[4];
    __shared__ uint64_t ends[2][kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t b = blockIdx.x, P = a.max_pages, page = a.page_size;
    if (tid < 4) count[tid] = 0;
    grid_dependency_wait();
    launch_dependents();
    const int32_t *table = a.pages + (int64_t)b * P;
    int32_t rows = __ldg(a.rows + b);
    const int64_t cap = (int64_t)P * page;
    if (rows > cap) {
        if (tid == 0) report_error(a.err, kErrCheck, kKerEvict, 1);
        rows = (int32_t)cap;
    }
    rows = max(rows, 0);
    const int32_t used = (int32_t)(((int64_t)rows + page - 1) / page);

    // ---------------------------------------------------------- page weights
    // 2^lg lanes a page, four dims a lane where pages and rows start on 16 bytes
    const bool vec = page % 4 == 0 && (reinterpret_cast<uintptr_t>(a.mass) & 15u) == 0;
    const int units = vec ? page / 4 : page;
    int lg = 0;
    while (lg < 5 && (1 << lg) < units) ++lg;
    const int lanes = 1 << lg, li = lane & (lanes - 1), groups = kThreads >> lg;
    const float *mass = a.mass + (int64_t)b * cap;
    int32_t held_safe = 0, free_pages = 0;
    constexpr int kAhead = 4;  // pages a group sums at a time
    for (int32_t p0 = 0; p0 < used; p0 += groups * kAhead) {
        Sum s[kAhead];
        int32_t phys[kAhead];
        auto page_at = [&](int x) { return p0 + (x * groups) + (tid >> lg); };
#pragma unroll
        for (int x = 0; x < kAhead; ++x) phys[x] = page_at(x) < used ? table[page_at(x)] : -1;
        for (int u = li; u < units; u += lanes) {
            float4 v[kAhead];
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const int64_t r = (int64_t)page_at(x) * page + (vec ? 4 * u : u);
                v[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (r >= rows) continue;
                if (vec) {
                    v[x] = __ldg(reinterpret_cast<const float4 *>(mass + r));
                    if (r + 1 >= rows) v[x].y = 0.0f;
                    if (r + 2 >= rows) v[x].z = 0.0f;
                    if (r + 3 >= rows) v[x].w = 0.0f;
                } else {
                    v[x].x = __ldg(mass + r);
                }
            }
#pragma unroll
            for (int x = 0; x < kAhead; ++x)
            {
                s[x].add(v[x].x);
                if (!vec) continue;
                s[x].add(v[x].y);
                s[x].add(v[x].z);
                s[x].add(v[x].w);
            }
        }
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float hi = __shfl_xor_sync(0xffffffffu, s[x].hi, o);
                const float lo = __shfl_xor_sync(0xffffffffu, s[x].lo, o);
                if (o < lanes) {
                    s[x].add(hi);
                    s[x].lo += lo;
                }
            }
            const int32_t p = page_at(x);
            if (li == 0 && p < used) {
                const int64_t first = (int64_t)p * page, end = first + page;
                const bool safe = first < a.keep_first || end > max(rows - a.keep_last, 0);
                key[p] = phys[x] >= 0 && !safe ? s[x].key() : 0ull;
                held_safe += phys[x] >= 0 && safe;
                free_pages += phys[x] >= 0 && !safe;
            }
        }
    }
    held_safe = __reduce_add_sync(0xffffffffu, held_safe);
    free_pages = __reduce_add_sync(0xffffffffu, free_pages);
    __syncthreads();  // count is zero
    if (lane == 0) {
        if (held_safe) atomicAdd(&count[0], held_safe);
        if (free_pages) atomicAdd(&count[1], free_pages);
    }
    __syncthreads();
    held_safe = count[0];
    free_pages = count[1];
    const int32_t room = max(a.keep_pages - held_safe, 0);  // of the free pages, how many may stay

    // -------------------------------------------------------------- the border
    // Pages with keys above `border` stay, and the first `equal` at it.
    uint64_t border = ~0ull;
    int32_t equal = 0;
    if (free_pages <= room) {
        border = 0;  // all stay
    } else if (room > 0) {
        uint64_t lo = ~0ull, hi = 0;
        for (int32_t p = tid; p < used; p += kThreads)
            if (key[p]) {
                lo = min(lo, key[p]);
                hi = max(hi, key[p]);
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            lo = min(lo, (uint64_t)__shfl_xor_sync(0xffffffffu, lo, o));
            hi = max(hi, (uint64_t)__shfl_xor_sync(0xffffffffu, hi, o));
        }
        if (lane == 0) {
            ends[0][warp] = lo;
            ends[1][warp] = hi;
        }
        __syncthreads();
        if (tid < 4) count[tid] = 0;
        lo = ends[0][lane];
        hi = ends[1][lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            lo = min(lo, (uint64_t)__shfl_xor_sync(0xffffffffu, lo, o));
            hi = max(hi, (uint64_t)__shfl_xor_sync(0xffffffffu, hi, o));
        }
        __syncthreads();
        // at least `room` keys lie at lo or above, fewer above hi: the
        // room-th largest is in [lo, hi]
        bool exact = false;
        for (int step = 0; lo < hi && !exact; ++step) {
            const uint64_t mid = lo + (hi - lo) / 2 + 1;  // above lo
            int32_t n = 0;
            for (int32_t p = tid; p < used; p += kThreads) n += key[p] >= mid;
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0 && n) atomicAdd(&count[step & 3], n);
            if (tid == 0) count[(step + 2) & 3] = 0;
            __syncthreads();
            n = count[step & 3];
            if (n >= room) lo = mid;
            else hi = mid - 1;
            exact = n == room;
        }
        border = lo;
        if (exact) {
            equal = INT32_MAX;
        } else {  // how many of the keys at the border fit beside those above it
            int32_t n = 0;
            for (int32_t p = tid; p < used; p += kThreads) n += key[p] > border;
            int32_t total;
            block_exclusive_scan<kThreads>(n, scan, &total);
            equal = room - total;
        }
    }

    // ------------------------------------------------- the table and the list
    int32_t at_border = 0, listed = 0;  // in the pages before
    for (int32_t p0 = 0; p0 < P; p0 += kThreads) {
        const int32_t p = p0 + tid;
        const int32_t phys = p < P ? table[p] : -1;
        const uint64_t k = p < used ? key[p] : 0ull;
        bool gone = k != 0 && k < border;
        int32_t total;
        if (p0 < used && border != 0) {
            if (equal != INT32_MAX) {
                const int32_t rank = at_border + block_exclusive_scan<kThreads>(k == border && k, scan, &total);
                at_border += total;
                gone |= k == border && k && rank >= equal;
            }
            const int32_t at = listed + block_exclusive_scan<kThreads>(gone, scan, &total);
            listed += total;
            if (gone && a.freed) a.freed[(int64_t)b * P + at] = phys;
        }
        if (p < P) a.out[(int64_t)b * P + p] = gone ? CSA_PAGE_EVICTED : phys;
    }
    if (a.freed)
        for (int32_t p = listed + tid; p < P; p += kThreads) a.freed[(int64_t)b * P + p] = -1;
    if (a.n_freed && tid == 0) a.n_freed[b] = listed;
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs &a, cudaStream_t stream) {
    static PerContext pc;
    bool first;
    int dev;
    unsigned long long ctx;
    cudaError_t e = enter_context(pc, &first, &ctx, &dev);
    if (e != cudaSuccess) return e;
    if (first) {
        e = cudaFuncSetAttribute(cache_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kEvictMaxPages * 8);
        if (e != cudaSuccess) return e;
        entered_context(pc, dev, ctx);
    }
    return launch_early(cache_evict_kernel, dim3(a.batch), dim3(kThreads), (size_t)a.max_pages * 8, stream, a);
}

}  // namespace csa
