// Internal launch interface between the C ABI of the token operators
// (token_api.cpp) and their gfx950 kernels (rope_kernels.hip,
// attention_kernels.hip).  Not installed.
#pragma once

#include <cstddef>
#include <cstdint>

#include <hip/hip_runtime_api.h>

#include "bevpool_internal.h"

namespace bevpool {

constexpr int kMaxHeadDim = 256;
constexpr int kMaxRopeAxes = 4;

// Norm and rotation of head rows, shared by the forward, the backward and the
// append.
struct RopeParams {
    int32_t n_tokens, n_q_heads, n_k_heads, head_dim;
    int32_t dtype;
    const void *q, *k;             // forward inputs
    int64_t q_stride, k_stride;    // elements between tokens
    const void *q_weight, *k_weight;
    int32_t weight_dtype;
    float eps;
    int32_t half;                  // R / 2 rotated pairs
    int32_t n_axes;
    int32_t section_end[kMaxRopeAxes];   // first pair past each axis's section
    const int32_t *positions;      // [n_axes, n_tokens]
    const float *inv_freq;         // [half]
    int32_t adjacent;
    void *q_out, *k_out;
    int64_t q_out_stride, k_out_stride;
};

hipError_t run_qk_norm_rope(const RopeParams &p, hipStream_t stream);

struct RopeGradParams {
    RopeParams rope;               // q_out / k_out: dq / dk
    const void *dq_out, *dk_out;
    int64_t dq_out_stride, dk_out_stride;
    float *dq_weight, *dk_weight;
    float *partials;               // workspace
};

size_t rope_grad_workspace_bytes(int64_t n_tokens, int32_t n_q_heads, int32_t n_k_heads,
                                 int32_t head_dim);
hipError_t run_qk_norm_rope_backward(const RopeGradParams &p, hipStream_t stream);

// A batch of sequences over a cache of pages.
struct PagedParams {
    void *k_cache, *v_cache;       // [n_pages, heads, page_size, head_dim]
    int32_t cache_dtype;
    float k_scale, v_scale;
    int32_t n_pages, page_shift;   // page_size = 1 << page_shift
    const int32_t *q_offsets, *kv_lengths, *block_table;
    int32_t n_seqs, max_pages;
};

struct AppendParams {
    RopeParams rope;               // k_out unused
    const void *v;
    int64_t v_stride;
    PagedParams paged;
};

hipError_t run_kv_append(const AppendParams &p, hipStream_t stream);

struct AttnParams {
    const void *q;
    int64_t q_stride;
    int32_t dtype;
    int32_t n_tokens, n_q_heads, n_k_heads, head_dim;
    PagedParams paged;
    float scale;
    int32_t causal, window;
    void *out;
    int64_t out_stride;
    void *workspace;
};

size_t attention_workspace_bytes(int64_t n_tokens, int32_t n_seqs, int32_t n_q_heads,
                                 int32_t n_k_heads, int32_t head_dim, int32_t page_size,
                                 int32_t max_pages);
hipError_t run_paged_attention(const AttnParams &p, hipStream_t stream);

}  // namespace bevpool
