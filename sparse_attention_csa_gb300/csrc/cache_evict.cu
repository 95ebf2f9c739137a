// Pages of cached rows to give back, by the attention weight their rows
// received (sm_103a).
//
//     weight of page p = sum of mass[b, r] over its rows r in use
// Of the pages a sequence holds, those with rows that are to stay (the first,
// the last, and a page with room for the next ones) stay; of the others the
// heaviest stay while the budget lasts, the lower page among equals. The rest
// are marked in the table and listed.
//
// A cluster of blocks a sequence: they share its pages' sums, and the first one
// chooses. Groups of lanes sum a page each in three 32-bit words (roundings are
// found exactly by Knuth's two-sum), so that the order of the rows does not
// decide between two pages: 64-bit additions, of which the SM does two a clock,
// made it 44 us for 512 pages and 83 us for 64 sequences (13.3 and 22.3 us with
// two such words and one block a sequence). A group has one page at a time (two,
// with more loads on their way, took 0.5 and 2 us more).
// The border between staying and going: one histogram over the interval of the
// sums' keys, which is found with them, leaves a few sums in the border's bin,
// which are ranked among themselves. More than kCand of them (sums that are
// close, or equal, beside far ones) are parted by halving the interval and
// counting, 64 counts at most. (Halving alone took 8 to 20 counts of 500
// clocks.)
//
// Bound by the latency of its steps: 512 pages of 64 rows 4.9 us, 64 sequences
// of up to 1024 pages (8.6 MB) 11.1 us.
#include "common.cuh"
#include "internal.h"
#include "paged.h"

namespace csa {

namespace {

constexpr int kThreads = 512;
constexpr int kBins = 2 * kThreads;
constexpr int kCand = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kLargest = 3.402823466e38f;

// s = a + b rounded; returns what the rounding left out, exactly (Knuth).
__device__ __forceinline__ float two_sum(float a, float b, float *s) {
    const float t = a + b, c = t - a;
    *s = t;
    return (a - (t - c)) + (b - c);
}

__device__ __forceinline__ float next_below(float x) {  // x finite, not 0
    const int32_t u = __float_as_int(x);
    return __int_as_float(u > 0 ? u - 1 : u + 1);
}

// A sum in three words: the sum, what its roundings left out, and what the
// roundings of that did. With a `fold` after every four loads (16 rows) the
// second word stays below 17 2^-24 of the magnitudes' sum S, the third, lanes
// joined, below 2^-39. So the sum is exact for rows that are multiples of
// 2^-63 S, and otherwise each of a lane's rows rounds it by 2^-63 S at most.
// (In two words, pages of the same 64 rows in another order came out apart, and
// pages of 4096 rows held 37 bits. A fold after every load and every join: 5.2
// and 11.8 us in place of 4.9 and 11.1.)
struct Sum {
    float hi = 0.0f, lo = 0.0f, rest = 0.0f;
    __device__ __forceinline__ void add(float x) { rest += two_sum(lo, two_sum(hi, x, &hi), &lo); }
    __device__ __forceinline__ void add(float x, float y, float z) {  // another sum
        add(x);
        rest += two_sum(lo, y, &lo) + z;
    }
    __device__ __forceinline__ void fold() {
        float t;
        const float l = two_sum(hi, lo, &t);
        if (fabsf(t) <= kLargest) {  // an infinite or NaN sum keeps its first word
            hi = t;
            rest = two_sum(l, rest, &lo);
        }
    }
    // Order-preserving map to uint64, above 0; NaN above all. The first word is
    // the sum rounded down to 32 bits, the second what is left of it, rounded
    // down too: unlike rounding to the nearest, it has one result for a sum
    // whatever its three words.
    __device__ __forceinline__ uint64_t key() const {
        if (hi != hi) return ~0ull;
        float h = hi, l = 0.0f;
        if (fabsf(hi) <= kLargest && fabsf(lo) <= kLargest) {
            float t, r = two_sum(lo, rest, &t);
            l = two_sum(hi, t, &h);
            r = two_sum(l, r, &l);
            l = two_sum(h, l, &h);  // now |l| is half a unit of h at most, |r| half one of l
            r = two_sum(l, r, &l);
            if (l < 0.0f) {
                const float d = h;
                h = next_below(h);
                r += two_sum(d - h, l, &l);
                r = two_sum(l, r, &l);
            }
            if (r < 0.0f) l = next_below(l);
            if (!(fabsf(h) <= kLargest)) l = 0.0f;  // passed the largest number here
        }
        return (uint64_t)float_key(h) << 32 | float_key(l);
    }
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address of `p` in the cluster's first block.
__device__ __forceinline__ uint32_t in_first(const void *p) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)));
    return r;
}
__device__ __forceinline__ void to_first(uint64_t *p, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_first(p)), "l"(v) : "memory");
}
__device__ __forceinline__ void add_to_first(int32_t *p, int32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(in_first(p)), "r"(v) : "memory");
}
__device__ __forceinline__ void min_to_first(uint32_t *p, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.min.u32 [%0], %1;" ::"r"(in_first(p)), "r"(v) : "memory");
}
__device__ __forceinline__ void max_to_first(uint32_t *p, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(in_first(p)), "r"(v) : "memory");
}

__global__ void __launch_bounds__(kThreads, 2) cache_evict_kernel(const __grid_constant__ EvictArgs a, int32_t ranks) {
    extern __shared__ uint64_t key[];  // of each page: 0, stays or is not held
    __shared__ int32_t scan[kWarps + 1];
    __shared__ int32_t held[2], count[4];
    __shared__ uint32_t ends[2];  // first words of the smallest and the largest sum
    __shared__ int32_t bins[kBins];
    __shared__ uint64_t cand[kCand], border_s;
    __shared__ int32_t n_cand, equal_s, found[3];
    const int tid = threadIdx.x, lane = tid & 31;
    const int32_t rank = blockIdx.x % ranks;  // of the cluster
    const int32_t b = blockIdx.x / ranks, P = a.max_pages, page = a.page_size;
    if (tid < 4) count[tid] = 0;
    if (tid == 0) {
        held[0] = held[1] = 0;
        ends[0] = ~0u;
        ends[1] = 0;
        n_cand = 0;
    }
    bins[2 * tid] = bins[2 * tid + 1] = 0;
    cluster_sync();  // the first block's counts are zero, and it is there
    grid_dependency_wait();
    launch_dependents();
    const int32_t *table = a.pages + (int64_t)b * P;
    int32_t rows = __ldg(a.rows + b);
    const int64_t cap = (int64_t)P * page;
    if (rows > cap) {
        if (rank == 0 && tid == 0) report_error(a.err, kErrCheck, kKerEvict, 1);
        rows = (int32_t)cap;
    }
    rows = max(rows, 0);
    const int32_t used = (int32_t)(((int64_t)rows + page - 1) / page);

    // ---------------------------------------------------------- page weights
    // 2^lg lanes a page, with about four loads each (of four rows where pages and
    // mass start on 16 bytes): more lanes spend more on adding their sums up
    const bool vec = page % 4 == 0 && (reinterpret_cast<uintptr_t>(a.mass) & 15u) == 0;
    const int units = vec ? page / 4 : page;
    int lg = 0;
    while (lg < 5 && (4 << lg) < units) ++lg;
    const int lanes = 1 << lg, li = lane & (lanes - 1), groups = kThreads >> lg;
    const float *mass = a.mass + (int64_t)b * cap;
    int32_t held_safe = 0, free_pages = 0;
    uint32_t least = ~0u, most = 0;
    for (int32_t p0 = rank * groups; p0 < used; p0 += ranks * groups) {
        const int32_t p = p0 + (tid >> lg);
        const int32_t phys = p < used ? table[p] : -1;
        const int64_t first = (int64_t)p * page, end = first + page;
        // of the page's rows those in use, and the loads they take; both below
        // 2^31, so that a step of up to 32 past them stays in 32 bits
        const uint32_t n = p < used ? (uint32_t)min((int64_t)page, rows - first) : 0u;
        const uint32_t loads = vec ? (n + 3u) / 4u : n;
        Sum s;
        int i = 0;
#pragma unroll 4
        for (uint32_t u = li; u < loads; u += lanes) {
            if (vec) {
                const float4 v = __ldg(reinterpret_cast<const float4 *>(mass + first) + u);
                s.add(v.x);
                s.add(4u * u + 1u < n ? v.y : 0.0f);
                s.add(4u * u + 2u < n ? v.z : 0.0f);
                s.add(4u * u + 3u < n ? v.w : 0.0f);
            } else {
                s.add(__ldg(mass + first + u));
            }
            if ((++i & 3) == 0) s.fold();
        }
        for (int o = lanes >> 1; o > 0; o >>= 1) {
            const float hi = __shfl_xor_sync(0xffffffffu, s.hi, o);
            const float lo = __shfl_xor_sync(0xffffffffu, s.lo, o);
            s.add(hi, lo, __shfl_xor_sync(0xffffffffu, s.rest, o));
        }
        if (li == 0 && p < used) {
            const bool safe = first < a.keep_first || end > max(rows - a.keep_last, 0);
            uint64_t k = 0;
            if (phys >= 0 && !safe) {
                k = s.key();
                least = min(least, (uint32_t)(k >> 32));
                most = max(most, (uint32_t)(k >> 32));
                ++free_pages;
            }
            to_first(&key[p], k);
            held_safe += phys >= 0 && safe;
        }
    }
    held_safe = __reduce_add_sync(0xffffffffu, held_safe);
    free_pages = __reduce_add_sync(0xffffffffu, free_pages);
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
        if (held_safe) add_to_first(&held[0], held_safe);
        if (free_pages) {
            add_to_first(&held[1], free_pages);
            min_to_first(&ends[0], least);
            max_to_first(&ends[1], most);
        }
    }
    cluster_sync();
    if (rank != 0) return;
    held_safe = held[0];
    free_pages = held[1];
    const int32_t room = max(a.keep_pages - held_safe, 0);  // of the free pages, how many may stay

    // -------------------------------------------------------------- the border
    // Pages with keys above `border` stay, and the first `equal` at it (all, if
    // INT32_MAX).
    uint64_t border = ~0ull;
    int32_t equal = 0;
    if (free_pages <= room) {
        border = 0;  // all stay
    } else if (room > 0) {
        uint64_t lo = (uint64_t)ends[0] << 32, hi = (uint64_t)ends[1] << 32 | 0xffffffffu;
        // the bin of the room-th largest: equal keys share a bin, larger ones
        // never fall lower
        static_assert(kBins == 1 << 10, "bins");
        const int shift = max(64 - __clzll((long long)(hi - lo)) - 10, 0);
        for (int32_t p = tid; p < used; p += kThreads)
            if (key[p]) atomicAdd(&bins[(key[p] - lo) >> shift], 1);
        __syncthreads();
        {
            const int top = kBins - 1 - 2 * tid;  // two bins a thread, from the highest down
            const int32_t n0 = bins[top], n1 = bins[top - 1];
            int32_t total;
            const int32_t above = block_exclusive_scan<kThreads>(n0 + n1, scan, &total);
            if (above < room && room <= above + n0 + n1) {
                const bool first = room <= above + n0;
                found[0] = first ? top : top - 1;
                found[1] = first ? above : above + n0;
                found[2] = first ? n0 : n1;
            }
        }
        __syncthreads();
        const int32_t need = room - found[1], there = found[2];
        lo += (uint64_t)found[0] << shift;
        const uint64_t width = ((uint64_t)1 << shift) - 1;
        if (hi - lo > width) hi = lo + width;  // the last bin may reach past 2^64: a NaN's key is 2^64 - 1
        bool exact = need == there;
        if (!exact && there <= kCand) {
            for (int32_t p = tid; p < used; p += kThreads)
                if (key[p] >= lo && key[p] <= hi) cand[atomicAdd(&n_cand, 1)] = key[p];
            __syncthreads();
            if (tid < there) {
                const uint64_t mine = cand[tid];
                int32_t above = 0, from = 0;
                for (int32_t i = 0; i < there; ++i) {
                    above += cand[i] > mine;
                    from += cand[i] >= mine;
                }
                if (above < need && need <= from) {  // equal keys write the same
                    border_s = mine;
                    equal_s = need == from ? INT32_MAX : need - above;
                }
            }
            __syncthreads();
            border = border_s;
            equal = equal_s;
        } else {
            // at least `room` keys lie at lo or above, fewer above hi
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
    // as many blocks as their groups of lanes have pages, up to 8, while there are
    // three an SM at most (64 sequences: 4 blocks each 10.4 us, 8 each 10.9, with sums of two words)
    int sms, units = a.page_size % 4 == 0 ? a.page_size / 4 : a.page_size, lg = 0;
    e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    while (lg < 5 && (4 << lg) < units) ++lg;
    int ranks = 1;
    while (ranks < 8 && (int64_t)ranks * (kThreads >> lg) < a.max_pages && (int64_t)2 * ranks * a.batch <= 3 * sms)
        ranks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ranks * a.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)a.max_pages * 8;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, cache_evict_kernel, a, (int32_t)ranks);
}

}  // namespace csa
