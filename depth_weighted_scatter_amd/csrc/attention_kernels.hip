// Attention over a paged cache (gfx950).  See bevpool.h for the definition.
#include <hip/hip_runtime.h>

#include "token_device.h"

namespace bevpool {
namespace {

constexpr int kBlock = 256;
constexpr int kWavesPerBlock = kBlock / kLanes;
constexpr float kLog2e = 1.44269504088896340736f;

template <int DT>
__device__ __forceinline__ float element(const void *base, int64_t i)
{
    if constexpr (DT == kE4M3) {
        const int w = static_cast<const uint8_t *>(base)[i];
        return __builtin_amdgcn_cvt_f32_fp8(w, 0);
    } else {
        return float(static_cast<const typename Elem<DT>::type *>(base)[i]);
    }
}

// One wave for each (token, query head): keys one after the other, the lanes
// over the head's elements, running maximum and sum of the softmax.
template <int DT, int CDT>
__global__ __launch_bounds__(kBlock) void attend_rows(AttnParams p)
{
    using T = typename Elem<DT>::type;
    constexpr int kPer = kMaxHeadDim / kLanes;
    const PagedParams &g = p.paged;
    const int lane = int(threadIdx.x) & (kLanes - 1);
    const int64_t row = int64_t(blockIdx.x) * kWavesPerBlock + int(threadIdx.x) / kLanes;
    if (row >= int64_t(p.n_tokens) * p.n_q_heads) return;
    const int token = int(row / p.n_q_heads), head = int(row % p.n_q_heads);
    const int kv_head = head / (p.n_q_heads / p.n_k_heads);
    const auto off = [&](int i) { return int64_t(clip(g.q_offsets[i], 0, p.n_tokens)); };
    const int seq = count_upto(g.n_seqs, token, off);
    if (seq >= g.n_seqs || token < off(seq) || token >= off(seq + 1)) return;
    const int begin = int(off(seq)), end = int(off(seq + 1));
    const int64_t room = int64_t(g.max_pages) << g.page_shift;
    const int64_t len = g.kv_lengths[seq] < 0 ? 0 : (g.kv_lengths[seq] < room ? g.kv_lengths[seq] : room);
    const int64_t place = len - (end - begin) + (token - begin);
    int64_t last = p.causal ? (place < len - 1 ? place : len - 1) : len - 1;
    int64_t first = p.window > 0 ? place - p.window + 1 : 0;
    if (first < 0) first = 0;

    float q[kPer], o[kPer];
    const T *src = static_cast<const T *>(p.q) + int64_t(token) * p.q_stride + int64_t(head) * p.head_dim;
    for (int i = 0; i < kPer; ++i) {
        const int d = lane + i * kLanes;
        q[i] = d < p.head_dim ? float(src[d]) : 0.0f;
        o[i] = 0.0f;
    }
    float top = -INFINITY, sum = 0.0f;
    const float c = p.scale * g.k_scale * kLog2e;
    for (int64_t j = first; j <= last; ++j) {
        const int page = g.block_table[int64_t(seq) * g.max_pages + (j >> g.page_shift)];
        if (page < 0 || page >= g.n_pages) continue;
        const int64_t at = (((int64_t(page) * p.n_k_heads + kv_head) << g.page_shift) +
                            (j & ((1 << g.page_shift) - 1))) * p.head_dim;
        float s = 0.0f;
        for (int i = 0; i < kPer; ++i) {
            const int d = lane + i * kLanes;
            if (d < p.head_dim) s = fmaf(q[i], element<CDT>(g.k_cache, at + d), s);
        }
        for (int m = 32; m > 0; m /= 2) s += __shfl_xor(s, m);
        s *= c;
        const float new_top = fmaxf(top, s);
        const float base = new_top == -INFINITY ? 0.0f : new_top;
        const float keep = exp2f(top - base), w = exp2f(s - base);
        top = new_top;
        sum = sum * keep + w;
        for (int i = 0; i < kPer; ++i) {
            const int d = lane + i * kLanes;
            if (d < p.head_dim) o[i] = fmaf(w, element<CDT>(g.v_cache, at + d), o[i] * keep);
        }
    }
    const float f = sum == 0.0f ? 0.0f : g.v_scale / sum;
    T *dst = static_cast<T *>(p.out) + int64_t(token) * p.out_stride + int64_t(head) * p.head_dim;
    for (int i = 0; i < kPer; ++i) {
        const int d = lane + i * kLanes;
        if (d < p.head_dim) dst[d] = T(o[i] * f);
    }
}

}  // namespace

size_t attention_workspace_bytes(int64_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t)
{
    return 256;
}

hipError_t run_paged_attention(const AttnParams &p, hipStream_t stream)
{
    const int64_t rows = int64_t(p.n_tokens) * p.n_q_heads;
    const uint32_t blocks = uint32_t((rows + kWavesPerBlock - 1) / kWavesPerBlock);
    const bool e4m3 = p.paged.cache_dtype == kE4M3;
    if (p.dtype == kF16 && !e4m3)
        attend_rows<kF16, kF16><<<blocks, kBlock, 0, stream>>>(p);
    else if (p.dtype == kF16)
        attend_rows<kF16, kE4M3><<<blocks, kBlock, 0, stream>>>(p);
    else if (!e4m3)
        attend_rows<kBF16, kBF16><<<blocks, kBlock, 0, stream>>>(p);
    else
        attend_rows<kBF16, kE4M3><<<blocks, kBlock, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace bevpool
