// Walks the tiles of block-scaled appends on the host (append_walk.h) and prints the
// pieces.  In, for each batch: PER block_shift page_shift n_tokens n_seqs max_pages
// n_pages, then offsets, lengths and table.  Out: "tile token0 row0 count early kept"
// a piece, "end" a batch.
#include <cstdio>
#include <vector>

#include "append_walk.h"

using namespace bevpool;

template <int PER>
static void walk(const AppendParams &a)
{
    const PagedParams &g = a.paged;
    const int shift = g.block_shift;
    const int64_t tiles = (a.rope.n_tokens >> shift) + PER * int64_t(g.n_seqs);
    for (int64_t tile = 0; tile < tiles; ++tile) {
        int seq = 0;
        for (int i = 1; i <= g.n_seqs; ++i) seq += first_tile<PER>(token_offset(a, i), i, shift) <= tile;
        if (seq >= g.n_seqs) continue;
        pieces_of<PER>(a, seq, tile, [&](const Piece &c) {
            printf("%lld %lld %lld %d %d %d\n", (long long)tile, (long long)c.token0, (long long)c.row0, c.count,
                   c.early, int(c.kept));
        });
    }
    puts("end");
}

static bool read(std::vector<int32_t> &v, size_t n)
{
    v.resize(n);
    for (int32_t &x : v)
        if (scanf("%d", &x) != 1) return false;
    return true;
}

int main()
{
    int per, n_tokens, n_seqs, max_pages;
    AppendParams a{};
    PagedParams &g = a.paged;
    a.rope.n_k_heads = 1;
    while (scanf("%d %d %d %d %d %d %d", &per, &g.block_shift, &g.page_shift, &n_tokens, &n_seqs, &max_pages,
                 &g.n_pages) == 7) {
        std::vector<int32_t> off, len, table;
        if (!read(off, size_t(n_seqs) + 1) || !read(len, n_seqs) || !read(table, size_t(n_seqs) * max_pages))
            return 1;
        a.rope.n_tokens = n_tokens;
        g.n_seqs = n_seqs;
        g.max_pages = max_pages;
        g.q_offsets = off.data();
        g.kv_lengths = len.data();
        g.block_table = table.data();
        if (per == 1) walk<1>(a);
        else walk<2>(a);
    }
    return 0;
}
