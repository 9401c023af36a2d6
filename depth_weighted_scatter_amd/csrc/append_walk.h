// Which new tokens the tiles of a block-scaled append take, as scalar code without a
// launch around it (append_scaled_kernels.hip runs it; it runs on the host as well).
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

#include "token_internal.h"

namespace bevpool {

// New tokens of one block.
struct Piece {
    int64_t token0;       // first of them
    int64_t row0;         // the block's first slot, in rows of head 0
    int count, early;     // new tokens, at least one; places before them in the block
    bool kept;            // the block is on a page
};

// Where sequence i begins among the tokens that are there.
__host__ __device__ __forceinline__ int64_t token_offset(const AppendParams &a, int i)
{
    const int off = a.paged.q_offsets[i];
    return off < 0 ? 0 : (off < a.rope.n_tokens ? off : a.rope.n_tokens);
}

// Tiles of the launch, a block of tokens each: sequence s has those from
// off(s) / tokens + PER s on, and so at least n / tokens + PER for its n new
// tokens, which lie in at most n / tokens + 2 blocks.  With PER = 1 the last tile
// takes what is left; with 2 there is none left (and half of the tiles of
// sequences of few tokens are nobody's).
template <int PER>
__host__ __device__ __forceinline__ int64_t first_tile(int64_t off, int seq, int block_shift)
{
    return (off >> block_shift) + PER * int64_t(seq);
}

// Calls f(Piece) for the new tokens of a tile, of the last sequence that begins at it
// or before (the first one if none does).
template <int PER, typename F>
__host__ __device__ __forceinline__ void pieces_of(const AppendParams &a, int seq, int64_t tile, F f)
{
    const PagedParams &g = a.paged;
    const int shift = g.block_shift;
    const int64_t begin = token_offset(a, seq), end = token_offset(a, seq + 1);
    // tokens before the first sequence have tiles too, which are nobody's
    const int64_t nth = tile - first_tile<PER>(begin, seq, shift);
    if (begin >= end || nth < 0) return;
    const int64_t place0 = int64_t(g.kv_lengths[seq]) - g.q_offsets[seq + 1] + begin;
    const int64_t place_end = place0 + end - begin;
    int64_t block = (place0 >> shift) + nth;
    const int64_t block_end = ((place_end - 1) >> shift) + 1;
    const bool last_tile = tile + 1 == first_tile<PER>(end, seq + 1, shift);
    for (; block < block_end; ++block) {
        const int64_t from = block << shift, to = (block + 1) << shift;
        const int64_t lo = place0 > from ? place0 : from, hi = place_end < to ? place_end : to;
        Piece c;
        c.count = int(hi - lo);
        c.early = int(lo - from);
        c.token0 = begin + lo - place0;
        int page = -1;
        if (lo >= 0 && lo < int64_t(g.max_pages) << g.page_shift)
            page = g.block_table[int64_t(seq) * g.max_pages + (lo >> g.page_shift)];
        c.kept = page >= 0 && page < g.n_pages;
        c.row0 = ((int64_t(c.kept ? page : 0) * a.rope.n_k_heads) << g.page_shift) +
                 (from & ((1 << g.page_shift) - 1));
        f(c);
        if (PER == 2 || !last_tile) return;
    }
}

}  // namespace bevpool
