"""The launch that adds the splits of an attention: as many blocks as the chip wants,
whatever the tiles (the rule compiled for the host; CPU, no GPU needed)."""
import os
import subprocess

import numpy as np
import pytest

from test_tokens_codegen import CSRC, HIPCC, ROOT

CUS = 256


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("join") / "join")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", f"-I{os.path.join(ROOT, 'include')}",
           f"-I{CSRC}", os.path.join(ROOT, "tests", "join_blocks_main.hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]

    def run(batches):
        text = "\n".join(" ".join(map(str, b)) for b in batches)
        r = subprocess.run([out], input=text, capture_output=True, text=True, timeout=60)
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return run


# scaled, tokens, sequences, heads, head_dim, page, pages: a token of many heads on one,
# short chunks over long contexts, wide heads
FEW_TILES = [(s, *b) for s in (0, 1) for b in [
    (1, 1, 64, 1, 128, 256, 512), (256, 1, 8, 2, 128, 64, 128), (16, 1, 32, 8, 128, 64, 512),
    (128, 2, 8, 2, 256, 64, 256)]]


@pytest.mark.parametrize("batch", FEW_TILES, ids=str)
def test_few_tiles_fill_the_chip(launches, batch):
    (tile_rows, tiles, splits, blocks), = launches([batch])
    assert splits > 4
    each = tiles * batch[4]
    # one more a tile would pass the chip, or the tile's 16 are there
    assert blocks == 16 or blocks * each <= CUS < (blocks + 1) * each


def test_blocks_of_any_batch(launches):
    """A tile has a block for every 64 rows, no more where tiles fill the chip, and at
    most 16; tiles of few rows have one, or four of many splits."""
    rng = np.random.default_rng(403)
    batches = []
    for _ in range(2000):
        hk, seqs = int(rng.choice([1, 2, 5, 8])), int(2 ** rng.uniform(0, 9))
        batches.append((int(rng.integers(0, 2)), int(seqs * 2 ** rng.uniform(0, 9)), seqs,
                        hk * int(rng.choice([1, 4, 8])), hk, int(rng.choice([64, 80, 128, 256])), 64,
                        int(2 ** rng.uniform(0, 12))))
    few = 0
    for (_, n, seqs, hq, hk, *_), (tile_rows, tiles, splits, blocks) in zip(batches, launches(batches)):
        if n * (hq // hk) <= 32 * seqs:
            few += 1
            assert blocks == (4 if splits >= 16 else 1)
            continue
        least = -(-tile_rows // 64)
        assert least <= blocks <= 16
        assert blocks == least or blocks * tiles * hk <= CUS
    assert 200 < few < 1800
