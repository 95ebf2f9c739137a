// C ABI of the rotation and of the paged-cache operators: host-side argument
// checks and launches. The operations and their errors are documented in
// include/csa.h.
#include <cmath>

#include "common.cuh"
#include "csa.h"
#include "internal.h"
#include "paged.h"

namespace {

csa_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA; }

bool misaligned(const void *p, uintptr_t bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }

int elem_size(csa_dtype_t d) { return d == CSA_F32 ? 4 : 2; }

bool known(csa_dtype_t d) { return d == CSA_BF16 || d == CSA_F32; }
bool known(csa_rope_layout_t l) { return l == CSA_ROPE_INTERLEAVED || l == CSA_ROPE_HALF; }

constexpr int32_t kMaxRopeDim = 1024;
constexpr int32_t kMaxKeys = 1 << 27;  // of a token in either cache: tile counts of many tokens stay in 32 bits

// Do [a, a + rows of `len` bytes every `sa`] and the same at b share a byte?
// Rows of two column ranges of one wider matrix (equal strides) do not.
bool overlaps(uintptr_t a, int64_t sa, uintptr_t b, int64_t sb, int64_t rows, int64_t len) {
    const uintptr_t ea = a + (uintptr_t)((rows - 1) * sa + len);
    const uintptr_t eb = b + (uintptr_t)((rows - 1) * sb + len);
    if (ea <= b || eb <= a) return false;
    if (sa != sb || rows == 1) return true;
    const int64_t d = (int64_t)((a < b ? b - a : a - b) % (uintptr_t)sa);
    return d < len || sa - d < len;
}

}  // namespace

extern "C" {

csa_status_t csa_rope_freqs(int32_t rope_dim, double theta, double factor, int32_t original_len,
                            double beta_fast, double beta_slow, double *inv_freq,
                            csa_stream_t stream) {
    if (!inv_freq) return CSA_ERR_NULL;
    if (rope_dim < 2 || (rope_dim & 1) || original_len < 0) return CSA_ERR_SHAPE;
    if (!std::isfinite(theta) || !(theta > 1.0) || !std::isfinite(factor) || !(factor >= 1.0))
        return CSA_ERR_UNSUPPORTED;
    if (original_len > 0 && (!std::isfinite(beta_fast) || !std::isfinite(beta_slow) ||
                             !(beta_slow > 0.0) || !(beta_fast >= beta_slow)))
        return CSA_ERR_UNSUPPORTED;
    csa::RopeFreqsArgs a;
    a.theta = theta;
    a.factor = factor;
    a.beta_fast = beta_fast;
    a.beta_slow = beta_slow;
    a.rope_dim = rope_dim;
    a.original_len = original_len;
    a.inv_freq = inv_freq;
    return from_cuda(csa::launch_rope_freqs(a, (cudaStream_t)stream));
}

csa_status_t csa_rope(const void *x, csa_dtype_t dtype, int64_t x_stride, const int32_t *positions,
                      const int32_t *cu_seqlens, int32_t batch, int32_t pos_stride,
                      const double *inv_freq, int32_t total_tokens, int32_t heads,
                      int32_t head_dim, int32_t rope_offset, int32_t rope_dim,
                      csa_rope_layout_t layout, float mscale, int32_t inverse, void *out,
                      int64_t out_stride, csa_stream_t stream) {
    if (total_tokens < 0 || batch < 0 || heads < 1 || head_dim < 1) return CSA_ERR_SHAPE;
    if (rope_dim < 2 || (rope_dim & 1) || rope_offset < 0 || rope_dim > head_dim ||
        rope_offset > head_dim - rope_dim)
        return CSA_ERR_SHAPE;
    const int64_t len = (int64_t)heads * head_dim;
    if (total_tokens > 1 && (x_stride < len || out_stride < len)) return CSA_ERR_SHAPE;
    if (!known(dtype) || !known(layout) || rope_dim > kMaxRopeDim || heads > 65535)
        return CSA_ERR_UNSUPPORTED;
    if (total_tokens == 0) return CSA_OK;  // nothing to do (empty buffers may be NULL)
    if (!x || !out || !inv_freq || (!positions && !cu_seqlens)) return CSA_ERR_NULL;
    const int es = elem_size(dtype);
    if (misaligned(x, es) || misaligned(out, es)) return CSA_ERR_UNSUPPORTED;
    if (total_tokens == 1) x_stride = out_stride = len;
    if (x == out ? x_stride != out_stride
                 : overlaps((uintptr_t)x, x_stride * es, (uintptr_t)out, out_stride * es,
                            total_tokens, len * es))
        return CSA_ERR_UNSUPPORTED;
    csa_status_t st;
    int32_t *err = csa::device_error_word(&st);
    if (st != CSA_OK) return st;
    csa::RopeArgs a;
    a.x = x;
    a.out = out;
    a.positions = positions;
    a.cu = cu_seqlens;
    a.inv_freq = inv_freq;
    a.err = err;
    a.x_stride = x_stride;
    a.out_stride = out_stride;
    a.T = total_tokens;
    a.H = heads;
    a.D = head_dim;
    a.off = rope_offset;
    a.n = rope_dim;
    a.batch = batch;
    a.pos_stride = pos_stride;
    a.f32 = dtype == CSA_F32;
    a.half = layout == CSA_ROPE_HALF;
    a.inverse = inverse != 0;
    a.mscale = mscale;
    return from_cuda(csa::launch_rope(a, (cudaStream_t)stream));
}

csa_status_t csa_cache_append(const void *rows, csa_dtype_t dtype, int64_t row_stride,
                              const int32_t *row_seq, const int32_t *row_pos,
                              const int32_t *pages, int32_t batch, int32_t max_pages,
                              int32_t num_pages, int32_t page_size, int32_t total_rows,
                              int32_t width, const double *inv_freq, int32_t rope_offset,
                              int32_t rope_dim, csa_rope_layout_t layout, float mscale,
                              int32_t pos_stride, csa_bf16_t *cache, csa_stream_t stream) {
    if (total_rows < 0 || batch < 0 || max_pages < 0 || num_pages < 0 || page_size < 1 || width < 1)
        return CSA_ERR_SHAPE;
    if (rope_dim < 0 || (rope_dim & 1) || rope_offset < 0 || rope_dim > width ||
        rope_offset > width - rope_dim)
        return CSA_ERR_SHAPE;
    if (total_rows > 1 && row_stride < width) return CSA_ERR_SHAPE;
    if (!row_seq && total_rows > batch) return CSA_ERR_SHAPE;
    if (!known(dtype) || !known(layout) || rope_dim > kMaxRopeDim) return CSA_ERR_UNSUPPORTED;
    if (total_rows == 0) return CSA_OK;  // nothing to do (empty buffers may be NULL)
    if (!rows || !row_pos || !pages || !cache || (rope_dim > 0 && !inv_freq)) return CSA_ERR_NULL;
    if (misaligned(rows, elem_size(dtype)) || misaligned(cache, 2)) return CSA_ERR_UNSUPPORTED;
    csa_status_t st;
    int32_t *err = csa::device_error_word(&st);
    if (st != CSA_OK) return st;
    csa::AppendArgs a;
    a.rows = rows;
    a.row_seq = row_seq;
    a.row_pos = row_pos;
    a.pages = pages;
    a.inv_freq = inv_freq;
    a.cache = reinterpret_cast<__nv_bfloat16 *>(cache);
    a.err = err;
    a.row_stride = total_rows == 1 ? width : row_stride;
    a.T = total_rows;
    a.D = width;
    a.off = rope_offset;
    a.n = rope_dim;
    a.pos_stride = pos_stride;
    a.batch = batch;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.f32 = dtype == CSA_F32;
    a.half = layout == CSA_ROPE_HALF;
    a.mscale = mscale;
    return from_cuda(csa::launch_cache_append(a, (cudaStream_t)stream));
}

size_t csa_indexer_topk_paged_workspace_size(int32_t total_tokens, int32_t max_rows,
                                             int32_t index_heads, int32_t index_dim, int32_t topk) {
    (void)index_heads;
    (void)index_dim;
    (void)topk;
    if (total_tokens <= 0 || max_rows < 0) return 0;
    return csa::indexer_paged_workspace_bytes(total_tokens, max_rows);
}

csa_status_t csa_indexer_topk_paged(const csa_bf16_t *q, const csa_bf16_t *k_cache, const float *w,
                                    const int32_t *pages, const int32_t *q_seq,
                                    const int32_t *q_pos, int32_t batch, int32_t total_tokens,
                                    int32_t index_heads, int32_t index_dim, int32_t num_pages,
                                    int32_t page_size, int32_t max_pages, int32_t cmp_ratio,
                                    int32_t topk, int32_t *topk_idx, float *topk_val,
                                    void *workspace, size_t workspace_bytes, csa_stream_t stream) {
    if (total_tokens < 0 || batch < 0 || num_pages < 0 || max_pages < 0 || page_size < 1 || topk < 1)
        return CSA_ERR_SHAPE;
    const int64_t max_rows = (int64_t)max_pages * page_size;
    if (max_rows > INT32_MAX || (!q_seq && total_tokens > batch)) return CSA_ERR_SHAPE;
    if (index_dim != 64 && index_dim != 128) return CSA_ERR_UNSUPPORTED;
    if (index_heads < 1 || index_heads > 64) return CSA_ERR_UNSUPPORTED;
    if (cmp_ratio < 2 || total_tokens > 65535) return CSA_ERR_UNSUPPORTED;
    if (total_tokens == 0) return CSA_OK;  // nothing to do (empty buffers may be NULL)
    if (!q || !w || !q_pos || !topk_idx) return CSA_ERR_NULL;
    if (max_rows > 0 && num_pages > 0 && (!k_cache || !pages)) return CSA_ERR_NULL;
    const size_t need = csa::indexer_paged_workspace_bytes(total_tokens, max_rows);
    if (need > 0 && (!workspace || workspace_bytes < need || misaligned(workspace, 256)))
        return CSA_ERR_WORKSPACE;
    if (misaligned(q, 16) || misaligned(k_cache, 16)) return CSA_ERR_UNSUPPORTED;
    csa_status_t st;
    int32_t *err = csa::device_error_word(&st);
    if (st != CSA_OK) return st;
    csa::IndexerPagedArgs a;
    a.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    a.k = {reinterpret_cast<const __nv_bfloat16 *>(k_cache), pages, num_pages, page_size,
           k_cache && pages ? max_pages : 0};
    a.w = w;
    a.q_seq = q_seq;
    a.q_pos = q_pos;
    a.topk_idx = topk_idx;
    a.topk_val = topk_val;
    a.scores = static_cast<float *>(workspace);
    a.err = err;
    a.T = total_tokens;
    a.Hi = index_heads;
    a.Di = index_dim;
    a.batch = batch;
    a.cmp_ratio = cmp_ratio;
    a.topk = topk;
    a.max_rows = a.k.max_pages > 0 ? (int32_t)max_rows : 0;
    a.wait_ns = csa::pipeline_wait_limit_ns();
    return from_cuda(csa::launch_indexer_topk_paged(a, (cudaStream_t)stream));
}

size_t csa_sparse_mla_paged_workspace_size(int32_t total_tokens, int32_t heads) {
    if (total_tokens <= 0 || heads < 1) return 0;
    return csa::mla_paged_workspace_bytes(total_tokens, heads);
}

csa_status_t csa_sparse_mla_paged(
    const csa_bf16_t *q, const csa_bf16_t *ori_cache, const csa_bf16_t *cmp_cache,
    const int32_t *cmp_sparse_indices, const int32_t *ori_pages, const int32_t *cmp_pages,
    const int32_t *q_seq, const int32_t *q_pos, int32_t batch, int32_t total_tokens, int32_t heads,
    int32_t head_dim, int32_t ori_num_pages, int32_t ori_page_size, int32_t ori_max_pages,
    int32_t cmp_num_pages, int32_t cmp_page_size, int32_t cmp_max_pages, int32_t topk,
    const float *sinks, float softmax_scale, int32_t cmp_ratio, int32_t ori_win_left,
    int32_t ori_win_right, csa_bf16_t *out, float *softmax_lse, int32_t return_softmax_lse,
    void *workspace, size_t workspace_bytes, csa_stream_t stream) {
    const bool use_cmp = cmp_cache != nullptr;
    if (batch < 0 || total_tokens < 0 || heads < 1 || ori_win_left < 0 || ori_num_pages < 0 ||
        ori_max_pages < 0 || ori_page_size < 1 ||
        (int64_t)ori_max_pages * ori_page_size > INT32_MAX)
        return CSA_ERR_SHAPE;
    if (use_cmp && (cmp_num_pages < 0 || cmp_max_pages < 0 || cmp_page_size < 1 ||
                    (int64_t)cmp_max_pages * cmp_page_size > INT32_MAX))
        return CSA_ERR_SHAPE;
    if (use_cmp && cmp_sparse_indices && topk < 1) return CSA_ERR_SHAPE;
    if (!q_seq && total_tokens > batch) return CSA_ERR_SHAPE;
    if (total_tokens > 0) {  // empty buffers may be NULL
        if (!q || !ori_cache || !ori_pages || !q_pos || !out) return CSA_ERR_NULL;
        if (return_softmax_lse && !softmax_lse) return CSA_ERR_NULL;
        if (use_cmp && !cmp_pages) return CSA_ERR_NULL;
    }
    if (head_dim != 512 || heads > 64 || ori_win_right != 0) return CSA_ERR_UNSUPPORTED;
    if (use_cmp && cmp_ratio < 2) return CSA_ERR_UNSUPPORTED;
    if (ori_win_left >= kMaxKeys ||
        (use_cmp && (cmp_sparse_indices ? topk : cmp_max_pages * cmp_page_size) > kMaxKeys))
        return CSA_ERR_UNSUPPORTED;
    if (misaligned(q, 16) || misaligned(ori_cache, 16) || misaligned(out, 16) ||
        (use_cmp && misaligned(cmp_cache, 16)))
        return CSA_ERR_UNSUPPORTED;
    if (total_tokens == 0) return CSA_OK;
    const size_t need = csa::mla_paged_workspace_bytes(total_tokens, heads);
    if (!workspace || workspace_bytes < need || misaligned(workspace, 256)) return CSA_ERR_WORKSPACE;
    csa_status_t st;
    int32_t *err = csa::device_error_word(&st);
    if (st != CSA_OK) return st;
    csa::MlaPagedArgs a;
    a.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    a.ori = {reinterpret_cast<const __nv_bfloat16 *>(ori_cache), ori_pages, ori_num_pages,
             ori_page_size, ori_max_pages};
    a.cmp = {reinterpret_cast<const __nv_bfloat16 *>(cmp_cache), cmp_pages, cmp_num_pages,
             cmp_page_size, cmp_max_pages};
    a.idx = use_cmp ? cmp_sparse_indices : nullptr;
    a.q_seq = q_seq;
    a.q_pos = q_pos;
    a.sinks = sinks;
    a.out = reinterpret_cast<__nv_bfloat16 *>(out);
    a.lse = return_softmax_lse ? softmax_lse : nullptr;
    a.workspace = workspace;
    a.err = err;
    a.T = total_tokens;
    a.H = heads;
    a.batch = batch;
    a.topk = a.idx ? topk : 0;
    a.cmp_ratio = use_cmp ? cmp_ratio : 1;
    a.window = ori_win_left + 1;
    a.softmax_scale = softmax_scale;
    a.wait_ns = csa::pipeline_wait_limit_ns();
    return from_cuda(csa::launch_sparse_mla_paged(a, (cudaStream_t)stream));
}

}  // extern "C"
