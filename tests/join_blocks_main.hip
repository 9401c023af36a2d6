// Prints how attention over splits is launched: in, for each batch, scaled n_tokens
// n_seqs n_q_heads n_k_heads head_dim page_size max_pages; out tile_rows tiles splits and
// the blocks that join a tile.
#include <cstdio>

#include "attention_device.h"

int main()
{
    using namespace bevpool;
    long long n;
    int scaled, seqs, hq, hk, dim, page, pages;
    while (scanf("%d %lld %d %d %d %d %d %d", &scaled, &n, &seqs, &hq, &hk, &dim, &page, &pages) == 8) {
        const Shape s = scaled ? shape_of<true>(n, seqs, hq, hk, dim, page, pages)
                               : shape_of<false>(n, seqs, hq, hk, dim, page, pages);
        printf("%d %lld %d %u\n", s.tile_rows, (long long)s.tiles, s.splits, join_blocks(s, n * hq, seqs, hk));
    }
    return 0;
}
