// C ABI of the token operators: host-side validation, then dispatch to the
// gfx950 kernels.  Declarations and the contract live in bevpool.h.
#include "bevpool.h"

#include <climits>
#include <cmath>
#include <cstdint>

#include "token_internal.h"

namespace {

using namespace bevpool;

constexpr int64_t kInt32Limit = int64_t(INT32_MAX);
static_assert(kMaxHeadDim == BEVPOOL_MAX_HEAD_DIM && kMaxRopeAxes == BEVPOOL_MAX_ROPE_AXES,
              "the kernels' limits are the header's");

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int token_bytes(int32_t dtype)
{
    switch (dtype) {
    case BEVPOOL_F32: return 4;
    case BEVPOOL_F16:
    case BEVPOOL_BF16: return 2;
    default: return 0;
    }
}

// Sizes every call checks: token and head counts and the head width.  Heads
// may be 0 where the caller allows it.
int check_sizes(int64_t n_tokens, int32_t n_q_heads, int32_t n_k_heads, int32_t head_dim)
{
    if (n_tokens < 0 || n_q_heads < 0 || n_k_heads < 0 || head_dim <= 0)
        return BEVPOOL_ERR_INVALID_ARG;
    if (head_dim % 16 != 0 || head_dim > kMaxHeadDim) return BEVPOOL_ERR_UNSUPPORTED;
    // heads are bounded first, so that no product wraps; the last bound keeps a
    // launch's threads (at most n_tokens * head_dim / 8) within the 32 bits of a grid
    const int64_t heads = int64_t(n_q_heads) + 2 * int64_t(n_k_heads);
    if (n_tokens > kInt32Limit || heads > kInt32Limit || n_tokens * heads > kInt32Limit ||
        n_tokens * head_dim > (int64_t(1) << 34))
        return BEVPOOL_ERR_OVERFLOW;
    return BEVPOOL_OK;
}

// One token tensor [n_tokens, heads, head_dim]: there, aligned, and with a
// stride that covers its heads and keeps rows 16-byte aligned.
int check_rows(const void *x, int64_t stride, int32_t heads, int32_t head_dim, int bytes)
{
    if (!x || !aligned(x, 16) || stride < int64_t(heads) * head_dim) return BEVPOOL_ERR_INVALID_ARG;
    if (stride > (int64_t(1) << 31)) return BEVPOOL_ERR_OVERFLOW;
    return (stride * bytes) % 16 != 0 ? BEVPOOL_ERR_INVALID_ARG : BEVPOOL_OK;
}

// Norm and rotation arguments; fills the fields of p that do not name token
// tensors.
int check_rope(int32_t dtype, int64_t n_tokens, int32_t n_q_heads, int32_t n_k_heads,
               int32_t head_dim, const void *q_weight, const void *k_weight, int32_t weight_dtype,
               float eps, const int32_t *positions, int32_t n_axes, const int32_t *h_sections,
               const float *inv_freq, int32_t layout, RopeParams &p)
{
    const int st = check_sizes(n_tokens, n_q_heads, n_k_heads, head_dim);
    if (st != BEVPOOL_OK) return st;
    if (n_axes < 0 || n_axes > kMaxRopeAxes || (n_axes > 0 && !h_sections)) return BEVPOOL_ERR_INVALID_ARG;
    if (layout != BEVPOOL_ROPE_HALVES && layout != BEVPOOL_ROPE_ADJACENT) return BEVPOOL_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || std::isinf(eps)) return BEVPOOL_ERR_INVALID_ARG;
    if ((q_weight || k_weight) && weight_dtype != dtype && weight_dtype != BEVPOOL_F32)
        return BEVPOOL_ERR_UNSUPPORTED;
    const int wb = weight_dtype == BEVPOOL_F32 ? 4 : 2;
    if ((q_weight && !aligned(q_weight, uintptr_t(wb))) || (k_weight && !aligned(k_weight, uintptr_t(wb))))
        return BEVPOOL_ERR_INVALID_ARG;
    p = RopeParams{};
    int64_t half = 0;
    for (int i = 0; i < n_axes; ++i) {
        if (h_sections[i] < 0) return BEVPOOL_ERR_INVALID_ARG;
        half += h_sections[i];
        p.section_end[i] = int32_t(half < kInt32Limit ? half : kInt32Limit);
    }
    if (2 * half > head_dim || half % 8 != 0) return BEVPOOL_ERR_UNSUPPORTED;
    if (half > 0 && n_tokens > 0 &&
        (!positions || !inv_freq || !aligned(positions, 4) || !aligned(inv_freq, 4)))
        return BEVPOOL_ERR_INVALID_ARG;
    p.n_tokens = int32_t(n_tokens);
    p.n_q_heads = n_q_heads;
    p.n_k_heads = n_k_heads;
    p.head_dim = head_dim;
    p.dtype = dtype;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.weight_dtype = weight_dtype;
    p.eps = eps;
    p.half = int32_t(half);
    p.n_axes = n_axes;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.adjacent = layout == BEVPOOL_ROPE_ADJACENT;
    return BEVPOOL_OK;
}

// Of the scores: far enough from fp32's ends that the distance at which the
// softmax's reference moves, 8 / scale, is finite.
bool good_scale(float s) { return s >= 0x1p-96f && s <= 0x1p96f; }

// far enough from fp32's ends that reciprocals and products stay normal
bool good_cache_scale(float s) { return s >= 0x1p-64f && s <= 0x1p64f; }

// Cache, page table and batch arrays; fills p.
int check_paged(int32_t dtype, int32_t n_k_heads, int64_t n_tokens,
                const void *k_cache, const void *v_cache, int32_t cache_dtype, float k_scale,
                float v_scale, int64_t n_pages, int32_t page_size, const int32_t *q_offsets,
                const int32_t *kv_lengths, int32_t n_seqs, const int32_t *block_table,
                int32_t max_pages, PagedParams &p)
{
    if (dtype != BEVPOOL_F16 && dtype != BEVPOOL_BF16) return BEVPOOL_ERR_UNSUPPORTED;
    if (cache_dtype != dtype && cache_dtype != BEVPOOL_FP8_E4M3) return BEVPOOL_ERR_UNSUPPORTED;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0)
        return BEVPOOL_ERR_UNSUPPORTED;
    if (n_k_heads <= 0 || n_seqs < 0 || max_pages < 0 || n_pages <= 0) return BEVPOOL_ERR_INVALID_ARG;
    if (n_seqs > (1 << 24) || n_pages > kInt32Limit || int64_t(max_pages) * page_size > (1 << 30) ||
        int64_t(n_seqs) * max_pages > kInt32Limit || n_pages * page_size > kInt32Limit)
        return BEVPOOL_ERR_OVERFLOW;
    if (cache_dtype == BEVPOOL_FP8_E4M3 && (!good_cache_scale(k_scale) || !good_cache_scale(v_scale)))
        return BEVPOOL_ERR_INVALID_ARG;
    p = PagedParams{};
    p.k_cache = const_cast<void *>(k_cache);
    p.v_cache = const_cast<void *>(v_cache);
    p.cache_dtype = cache_dtype;
    p.k_scale = cache_dtype == BEVPOOL_FP8_E4M3 ? k_scale : 1.0f;
    p.v_scale = cache_dtype == BEVPOOL_FP8_E4M3 ? v_scale : 1.0f;
    p.n_pages = int32_t(n_pages);
    p.page_shift = __builtin_ctz(uint32_t(page_size));
    p.q_offsets = q_offsets;
    p.kv_lengths = kv_lengths;
    p.block_table = block_table;
    p.n_seqs = n_seqs;
    p.max_pages = max_pages;
    if (n_tokens == 0 || n_seqs == 0) return BEVPOOL_OK;     // nothing is read or written
    if (!k_cache || !v_cache || !q_offsets || !kv_lengths || (!block_table && max_pages > 0))
        return BEVPOOL_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q_offsets, 4) ||
        !aligned(kv_lengths, 4) || !aligned(block_table, 4))
        return BEVPOOL_ERR_INVALID_ARG;
    return BEVPOOL_OK;
}

int status_of(hipError_t e) { return e == hipSuccess ? BEVPOOL_OK : BEVPOOL_ERR_HIP; }

}  // namespace

extern "C" {

int bevpool_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                         int32_t dtype, int64_t n_tokens, int32_t n_q_heads, int32_t n_k_heads,
                         int32_t head_dim, const void *q_weight, const void *k_weight,
                         int32_t weight_dtype, float eps, const int32_t *positions,
                         int32_t n_axes, const int32_t *h_sections, const float *inv_freq,
                         int32_t layout, void *q_out, int64_t q_out_stride, void *k_out,
                         int64_t k_out_stride, hipStream_t stream)
{
    RopeParams p;
    const int bytes = token_bytes(dtype);
    if (bytes == 0) return BEVPOOL_ERR_UNSUPPORTED;
    int st = check_rope(dtype, n_tokens, n_q_heads, n_k_heads, head_dim, q_weight, k_weight,
                        weight_dtype, eps, positions, n_axes, h_sections, inv_freq, layout, p);
    if (st != BEVPOOL_OK) return st;
    if (n_q_heads <= 0) return BEVPOOL_ERR_INVALID_ARG;
    if (n_tokens == 0) return BEVPOOL_OK;
    if ((st = check_rows(q, q_stride, n_q_heads, head_dim, bytes)) != BEVPOOL_OK ||
        (st = check_rows(q_out, q_out_stride, n_q_heads, head_dim, bytes)) != BEVPOOL_OK)
        return st;
    if (n_k_heads > 0 &&
        ((st = check_rows(k, k_stride, n_k_heads, head_dim, bytes)) != BEVPOOL_OK ||
         (st = check_rows(k_out, k_out_stride, n_k_heads, head_dim, bytes)) != BEVPOOL_OK))
        return st;
    p.q = q;
    p.k = k;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out = q_out;
    p.k_out = k_out;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    return status_of(run_qk_norm_rope(p, stream));
}

size_t bevpool_qk_norm_rope_backward_workspace_size(int64_t n_tokens, int32_t n_q_heads,
                                                    int32_t n_k_heads, int32_t head_dim)
{
    if (check_sizes(n_tokens, n_q_heads, n_k_heads, head_dim) != BEVPOOL_OK || n_q_heads <= 0)
        return 0;
    return rope_grad_workspace_bytes(n_tokens, n_q_heads, n_k_heads, head_dim);
}

int bevpool_qk_norm_rope_backward(const void *dq_out, int64_t dq_out_stride, const void *dk_out,
                                  int64_t dk_out_stride, const void *q, int64_t q_stride,
                                  const void *k, int64_t k_stride, int32_t dtype,
                                  int64_t n_tokens, int32_t n_q_heads, int32_t n_k_heads,
                                  int32_t head_dim, const void *q_weight, const void *k_weight,
                                  int32_t weight_dtype, float eps, const int32_t *positions,
                                  int32_t n_axes, const int32_t *h_sections,
                                  const float *inv_freq, int32_t layout, void *dq,
                                  int64_t dq_stride, void *dk, int64_t dk_stride,
                                  float *dq_weight, float *dk_weight, void *workspace,
                                  size_t workspace_bytes, hipStream_t stream)
{
    RopeGradParams g{};
    RopeParams &p = g.rope;
    const int bytes = token_bytes(dtype);
    if (bytes == 0) return BEVPOOL_ERR_UNSUPPORTED;
    int st = check_rope(dtype, n_tokens, n_q_heads, n_k_heads, head_dim, q_weight, k_weight,
                        weight_dtype, eps, positions, n_axes, h_sections, inv_freq, layout, p);
    if (st != BEVPOOL_OK) return st;
    if (n_q_heads <= 0) return BEVPOOL_ERR_INVALID_ARG;
    // no key heads: a given gradient of their weight becomes zeros
    if (n_k_heads == 0 && !dk_weight) p.k_weight = nullptr;
    if ((p.q_weight && (!dq_weight || !aligned(dq_weight, 4))) ||
        (p.k_weight && (!dk_weight || !aligned(dk_weight, 4))))
        return BEVPOOL_ERR_INVALID_ARG;
    if (n_tokens > 0) {
        if ((st = check_rows(dq_out, dq_out_stride, n_q_heads, head_dim, bytes)) != BEVPOOL_OK ||
            (st = check_rows(dq, dq_stride, n_q_heads, head_dim, bytes)) != BEVPOOL_OK)
            return st;
        if (p.q_weight && (st = check_rows(q, q_stride, n_q_heads, head_dim, bytes)) != BEVPOOL_OK)
            return st;
        if (n_k_heads > 0) {
            if ((st = check_rows(dk_out, dk_out_stride, n_k_heads, head_dim, bytes)) != BEVPOOL_OK ||
                (st = check_rows(dk, dk_stride, n_k_heads, head_dim, bytes)) != BEVPOOL_OK)
                return st;
            if (p.k_weight && (st = check_rows(k, k_stride, n_k_heads, head_dim, bytes)) != BEVPOOL_OK)
                return st;
        }
    }
    if (!workspace) return BEVPOOL_ERR_INVALID_ARG;
    if (!aligned(workspace, 256) ||
        workspace_bytes < rope_grad_workspace_bytes(n_tokens, n_q_heads, n_k_heads, head_dim))
        return BEVPOOL_ERR_WORKSPACE;
    p.q = q;
    p.k = k;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out = dq;
    p.k_out = dk;
    p.q_out_stride = dq_stride;
    p.k_out_stride = dk_stride;
    g.dq_out = dq_out;
    g.dk_out = dk_out;
    g.dq_out_stride = dq_out_stride;
    g.dk_out_stride = dk_out_stride;
    g.dq_weight = dq_weight;
    g.dk_weight = dk_weight;
    g.partials = static_cast<float *>(workspace);
    return status_of(run_qk_norm_rope_backward(g, stream));
}

int bevpool_kv_append(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                      const void *v, int64_t v_stride, int32_t dtype, int64_t n_tokens,
                      int32_t n_q_heads, int32_t n_k_heads, int32_t head_dim,
                      const void *q_weight, const void *k_weight, int32_t weight_dtype,
                      float eps, const int32_t *positions, int32_t n_axes,
                      const int32_t *h_sections, const float *inv_freq, int32_t layout,
                      void *q_out, int64_t q_out_stride, void *k_cache, void *v_cache,
                      int32_t cache_dtype, float k_scale, float v_scale, int64_t n_pages,
                      int32_t page_size, const int32_t *q_offsets, const int32_t *kv_lengths,
                      int32_t n_seqs, const int32_t *block_table, int32_t max_pages,
                      hipStream_t stream)
{
    AppendParams a{};
    RopeParams &p = a.rope;
    int st = check_rope(dtype, n_tokens, n_q_heads, n_k_heads, head_dim, q_weight, k_weight,
                        weight_dtype, eps, positions, n_axes, h_sections, inv_freq, layout, p);
    if (st != BEVPOOL_OK) return st;
    st = check_paged(dtype, n_k_heads, n_tokens, k_cache, v_cache, cache_dtype, k_scale,
                     v_scale, n_pages, page_size, q_offsets, kv_lengths, n_seqs, block_table,
                     max_pages, a.paged);
    if (st != BEVPOOL_OK) return st;
    if (n_tokens == 0 || n_seqs == 0) return BEVPOOL_OK;
    const int bytes = token_bytes(dtype);
    if ((st = check_rows(k, k_stride, n_k_heads, head_dim, bytes)) != BEVPOOL_OK ||
        (st = check_rows(v, v_stride, n_k_heads, head_dim, bytes)) != BEVPOOL_OK)
        return st;
    if (n_q_heads > 0 &&
        ((st = check_rows(q, q_stride, n_q_heads, head_dim, bytes)) != BEVPOOL_OK ||
         (st = check_rows(q_out, q_out_stride, n_q_heads, head_dim, bytes)) != BEVPOOL_OK))
        return st;
    p.q = q;
    p.k = k;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out = q_out;
    p.q_out_stride = q_out_stride;
    a.v = v;
    a.v_stride = v_stride;
    return status_of(run_kv_append(a, stream));
}

namespace {

// A launch has fewer than 2^32 threads, 512 a block: one block for every 128
// rows of a key head, and one for every sequence and key head.
bool too_many_blocks(int64_t n_tokens, int32_t n_seqs, int32_t n_q_heads, int32_t n_k_heads)
{
    return (n_tokens * (n_q_heads / n_k_heads) / 128 + n_seqs) * n_k_heads >= (1 << 23);
}

}  // namespace

size_t bevpool_paged_attention_workspace_size(int64_t n_tokens, int32_t n_seqs,
                                              int32_t n_q_heads, int32_t n_k_heads,
                                              int32_t head_dim, int32_t page_size,
                                              int32_t max_pages)
{
    if (check_sizes(n_tokens, n_q_heads, n_k_heads, head_dim) != BEVPOOL_OK || n_seqs < 0 ||
        n_q_heads <= 0 || n_k_heads <= 0 || n_q_heads % n_k_heads != 0 || max_pages < 0 ||
        n_seqs > (1 << 24) || page_size < 16 || page_size > 256 ||
        (page_size & (page_size - 1)) != 0 || int64_t(max_pages) * page_size > (1 << 30) ||
        too_many_blocks(n_tokens, n_seqs, n_q_heads, n_k_heads))
        return 0;
    return attention_workspace_bytes(n_tokens, n_seqs, n_q_heads, n_k_heads, head_dim, page_size,
                                     max_pages);
}

int bevpool_paged_attention(const void *q, int64_t q_stride, int32_t dtype, int64_t n_tokens,
                            int32_t n_q_heads, int32_t n_k_heads, int32_t head_dim,
                            const void *k_cache, const void *v_cache, int32_t cache_dtype,
                            float k_scale, float v_scale, int64_t n_pages, int32_t page_size,
                            const int32_t *q_offsets, const int32_t *kv_lengths, int32_t n_seqs,
                            const int32_t *block_table, int32_t max_pages, float scale,
                            int32_t causal, int32_t window, void *out, int64_t out_stride,
                            void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    AttnParams p{};
    int st = check_sizes(n_tokens, n_q_heads, n_k_heads, head_dim);
    if (st != BEVPOOL_OK) return st;
    st = check_paged(dtype, n_k_heads, n_tokens, k_cache, v_cache, cache_dtype, k_scale,
                     v_scale, n_pages, page_size, q_offsets, kv_lengths, n_seqs, block_table,
                     max_pages, p.paged);
    if (st != BEVPOOL_OK) return st;
    if (n_q_heads <= 0 || n_q_heads % n_k_heads != 0 || !good_scale(scale) ||
        !good_scale(scale * p.paged.k_scale) || window < 0 || (causal != 0 && causal != 1))
        return BEVPOOL_ERR_INVALID_ARG;
    if (too_many_blocks(n_tokens, n_seqs, n_q_heads, n_k_heads)) return BEVPOOL_ERR_OVERFLOW;
    if (n_tokens == 0 || n_seqs == 0) return BEVPOOL_OK;
    if ((st = check_rows(q, q_stride, n_q_heads, head_dim, 2)) != BEVPOOL_OK ||
        (st = check_rows(out, out_stride, n_q_heads, head_dim, 2)) != BEVPOOL_OK)
        return st;
    if (!workspace) return BEVPOOL_ERR_INVALID_ARG;
    if (!aligned(workspace, 256) ||
        workspace_bytes < attention_workspace_bytes(n_tokens, n_seqs, n_q_heads, n_k_heads,
                                                    head_dim, page_size, max_pages))
        return BEVPOOL_ERR_WORKSPACE;
    p.q = q;
    p.q_stride = q_stride;
    p.dtype = dtype;
    p.n_tokens = int32_t(n_tokens);
    p.n_q_heads = n_q_heads;
    p.n_k_heads = n_k_heads;
    p.head_dim = head_dim;
    p.scale = scale;
    p.causal = causal;
    p.window = window;
    p.out = out;
    p.out_stride = out_stride;
    p.workspace = workspace;
    return status_of(run_paged_attention(p, stream));
}

}  // extern "C"
