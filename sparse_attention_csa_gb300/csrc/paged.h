// Internal launchers of the rotation and of the paged-cache operators. The
// arguments are already validated by paged_api.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "common.cuh"
#include "csa.h"
#include "tc_ptx.cuh"
#include "tmap.h"

namespace csa {

// Whether this is the first call of this place (a static of the caller's) in
// the current device's present context: a kernel's attributes are set once for
// each.
constexpr int kPagedDevices = 64;
struct PerContext {
    std::atomic<unsigned long long> seen[kPagedDevices];
};
inline cudaError_t enter_context(PerContext &pc, bool *first, unsigned long long *ctx, int *device) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kPagedDevices) return cudaErrorInvalidDevice;
    *device = dev;
    *ctx = current_context_id();
    *first = *ctx == 0 || pc.seen[dev].load(std::memory_order_acquire) != *ctx;
    return cudaSuccess;
}
inline void entered_context(PerContext &pc, int device, unsigned long long ctx) {
    pc.seen[device].store(ctx, std::memory_order_release);
}

// SMs of the current device, looked up once.
inline cudaError_t sm_count(int *sms) {
    static std::atomic<int> known[kPagedDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kPagedDevices) return cudaErrorInvalidDevice;
    *sms = known[dev].load(std::memory_order_relaxed);
    if (*sms == 0) {
        e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        known[dev].store(*sms, std::memory_order_relaxed);
    }
    return cudaSuccess;
}

struct RopeFreqsArgs {
    double theta, factor, beta_fast, beta_slow;
    int32_t rope_dim, original_len;
    double *inv_freq;  // [rope_dim / 2]
};

cudaError_t launch_rope_freqs(const RopeFreqsArgs &a, cudaStream_t stream);

struct RopeArgs {
    const void *x;             // [T, H, D], token stride x_stride
    void *out;                 // [T, H, D], token stride out_stride
    const int32_t *positions;  // [T] or nullptr
    const int32_t *cu;         // [batch+1] when positions is nullptr
    const double *inv_freq;    // [n / 2] radians per position
    int32_t *err;
    int64_t x_stride, out_stride;  // elements
    int32_t T, H, D, off, n, batch, pos_stride;
    int32_t f32, half, inverse;
    float mscale;
};

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream);

struct AppendArgs {
    const void *rows;         // [T, D], row stride row_stride
    const int32_t *row_seq;   // [T] or nullptr (row t belongs to sequence t)
    const int32_t *row_pos;   // [T], negative: skipped
    const int32_t *pages;     // [batch, max_pages]
    const double *inv_freq;   // [n / 2] or nullptr (n = 0)
    __nv_bfloat16 *cache;     // [num_pages, page_size, D]
    int32_t *err;
    int64_t row_stride;
    int32_t T, D, off, n, pos_stride;
    int32_t batch, max_pages, num_pages, page_size;
    int32_t f32, half;
    float mscale;
};

cudaError_t launch_cache_append(const AppendArgs &a, cudaStream_t stream);

// One paged row cache as the kernels see it.
struct PagedRows {
    const __nv_bfloat16 *base;  // [num_pages, page_size, width]
    const int32_t *pages;       // [batch, max_pages]
    int32_t num_pages, page_size, max_pages;
};

struct IndexerPagedArgs {
    const __nv_bfloat16 *q;  // [T, Hi, Di]
    PagedRows k;             // width Di
    const float *w;          // [T, Hi]
    const int32_t *q_seq;    // [T] or nullptr
    const int32_t *q_pos;    // [T]
    int32_t *topk_idx;       // [T, topk]
    float *topk_val;         // [T, topk] or nullptr
    float *scores;           // workspace: [T, row_pad] scores
    int32_t *err;
    int32_t T, Hi, Di, batch, cmp_ratio, topk, max_rows;
    int64_t row_pad;         // floats between two tokens' scores
    uint64_t wait_ns;
};

size_t indexer_paged_workspace_bytes(int32_t T, int64_t max_rows);
cudaError_t launch_indexer_topk_paged(IndexerPagedArgs a, cudaStream_t stream);

// Of a token in either cache: the kernels scan the tile counts of many tokens in
// 32 bits.
constexpr int32_t kMaxKeys = 1 << 27;

struct MlaPagedArgs {
    const __nv_bfloat16 *q;  // [T, H, 512]
    PagedRows ori;           // width 512
    PagedRows cmp;           // width 512; base nullptr: window only
    const int32_t *idx;      // [T, topk] or nullptr (every visible row)
    const int32_t *q_seq;    // [T] or nullptr
    const int32_t *q_pos;    // [T]
    const float *sinks;      // [H] or nullptr
    __nv_bfloat16 *out;      // [T, H, 512]
    float *lse;              // [T, H] or nullptr
    void *workspace;
    int32_t *err;
    int32_t T, H, batch, topk, cmp_ratio, window;
    float softmax_scale;
    uint64_t wait_ns;
};

size_t mla_paged_workspace_bytes(int32_t T, int32_t H);
cudaError_t launch_sparse_mla_paged(MlaPagedArgs a, cudaStream_t stream);
// cmp.base then points at rows of 384 bytes (q4.cuh)
cudaError_t launch_sparse_mla_paged_q4(MlaPagedArgs a, cudaStream_t stream);

constexpr int32_t kQ4Dims = 448;  // dims of a 512-wide row held in 4 bits (q4.cuh)

struct Q4RowsArgs {
    const void *rows;        // append: [T, 512], row stride row_stride
    __nv_bfloat16 *out;      // read: [T, 512]
    const int32_t *row_seq;  // [T] or nullptr (row t belongs to sequence t)
    const int32_t *row_pos;  // [T], negative: skipped (read: zeros)
    const int32_t *pages;    // [batch, max_pages]
    const double *inv_freq;  // [n / 2] or nullptr (n = 0)
    uint8_t *cache;          // [num_pages, page_size, 384]
    int32_t *err;
    int64_t row_stride;
    int32_t T, off, n, pos_stride;  // rotary dims [off, off + n), within the last 64
    int32_t batch, max_pages, num_pages, page_size;
    int32_t f32, half;
    float mscale;
};

cudaError_t launch_cache_append_q4(const Q4RowsArgs &a, cudaStream_t stream);
cudaError_t launch_cache_read_q4(const Q4RowsArgs &a, cudaStream_t stream);

struct MassArgs {
    const __nv_bfloat16 *q;  // [T, H, 512]
    const float *lse;        // [T, H]
    PagedRows cmp;           // 512 wide, or (q4) 384 bytes a row
    const int32_t *idx;      // [T, topk] or nullptr (every visible row)
    const int32_t *q_seq;    // [T] or nullptr
    const int32_t *q_pos;    // [T]
    const float *mass;       // [batch, max_rows] or nullptr (zeros)
    float *out;              // [batch, max_rows], may be mass
    float *weights;          // workspace: [T, slot_pad]
    int32_t *err;
    int64_t slot_pad;
    int32_t T, H, batch, topk, cmp_ratio, max_rows, q4;
    float softmax_scale;
    int32_t lg_unit, lg_part;  // fixed-point units of a weight of 1, parts of a unit: their log2
    uint64_t wait_ns;
};

int64_t mass_slot_pad(int64_t slots);
size_t mass_workspace_bytes(int32_t T, int64_t slots);
cudaError_t launch_attn_mass(MassArgs a, cudaStream_t stream);

constexpr int32_t kEvictMaxPages = 24576;  // a sequence's sums in shared memory

struct EvictArgs {
    const float *mass;     // [batch, max_pages * page_size]
    const int32_t *pages;  // [batch, max_pages]
    const int32_t *rows;   // [batch] rows in use
    int32_t *out;          // [batch, max_pages], may be pages
    int32_t *freed;        // [batch, max_pages] or nullptr
    int32_t *n_freed;      // [batch] or nullptr
    int32_t *err;
    int32_t batch, max_pages, page_size, keep_pages, keep_first, keep_last;
};

cudaError_t launch_cache_evict(const EvictArgs &a, cudaStream_t stream);

#ifdef __CUDACC__
// Row of the pool (in rows) holding logical row r of sequence b, or -1 when
// the table has no page for it or names one outside the pool.
__device__ __forceinline__ int64_t paged_row(const PagedRows &p, int32_t b, int32_t r) {
    const uint32_t pg = (uint32_t)r / (uint32_t)p.page_size;
    if (pg >= (uint32_t)p.max_pages) return -1;
    const int32_t phys = __ldg(p.pages + (int64_t)b * p.max_pages + pg);
    if ((uint32_t)phys >= (uint32_t)p.num_pages) return -1;
    return (int64_t)phys * p.page_size + (r - (int32_t)pg * p.page_size);
}

// Sequence of token t: -1 for a padding slot (negative position), -2 when the
// sequence number is outside the batch.
__device__ __forceinline__ int32_t paged_seq(const int32_t *q_seq, int32_t batch, int32_t t,
                                             int32_t pos) {
    const int32_t b = q_seq ? __ldg(q_seq + t) : t;  // not behind the position's load
    if (pos < 0) return -1;
    return (uint32_t)b < (uint32_t)batch ? b : -2;
}

// A kernel's waits on its own pipeline barriers: bounded, and none begins once
// one has given up (recorded in the device error word; M::abort tells the CTA).
template <class M, int32_t kKernel>
struct PipeWaits {
    M *m;
    int32_t *err;
    uint64_t limit;  // a wait gives up after this long
    __device__ __forceinline__ bool aborted() const {
        return *reinterpret_cast<volatile int32_t *>(&m->abort) != 0;
    }
    __device__ __forceinline__ void fail(int site) const {
        *reinterpret_cast<volatile int32_t *>(&m->abort) = 1;
        report_error(err, kErrTimeout, kKernel, site);
    }
    // false on timeout or when already aborted
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, int site) const {
        if (aborted()) return false;
        if (tc::mbar_wait(bar, parity, limit)) return true;
        fail(site);
        return false;
    }
};

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

// a / b, by a 32-bit division when both fit.
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}
#endif

}  // namespace csa
