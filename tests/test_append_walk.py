"""Which tokens the tiles of a block-scaled append take: the walk that its kernels
run, compiled for the host, against the oracle's places (CPU, no GPU needed)."""
import os
import subprocess

import numpy as np
import pytest

from oracle import tokens as ref
from test_tokens_codegen import CSRC, HIPCC, ROOT

INT32 = 2 ** 31


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("walk") / "walk")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", f"-I{os.path.join(ROOT, 'include')}",
           f"-I{CSRC}", os.path.join(ROOT, "tests", "append_walk_main.hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return out


def walk(program, batches):
    """For each batch, its pieces (tile, token0, row0, count, early, kept)."""
    words = []
    for per, block, page, n, off, kv, table, n_pages in batches:
        words += [per, block.bit_length() - 1, page.bit_length() - 1, n, len(kv), table.shape[1], n_pages,
                  *off, *kv, *table.reshape(-1)]
    r = subprocess.run([program], input=" ".join(str(int(w)) for w in words), capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0
    got = [[tuple(map(int, line.split())) for line in part.splitlines()]
           for part in r.stdout.split("end\n")[:-1]]
    assert len(got) == len(batches)
    return got


def table_of(rng, n_seqs, width, n_pages):
    """Pages of the pool, each once, some entries on none."""
    table = rng.permutation(max(n_pages, n_seqs * width))[:n_seqs * width].reshape(n_seqs, width)
    return np.where(rng.random(table.shape) < 0.1, -1, table).astype(np.int64)


def check(batch, pieces):
    per, block, page, n, off, kv, table, n_pages = batch
    seq, _ = ref.places(off, kv, table.shape[1], page, n)
    found = []
    for tile, token0, row0, count, early, kept in pieces:
        assert count > 0 and early >= 0 and early + count <= block, (batch, tile)
        assert 0 <= token0 and token0 + count <= n
        found += range(token0, token0 + count)
    # every token of a sequence once, and no other
    assert sorted(found) == [t for t in range(n) if seq[t] >= 0]
    on = {(row0, early, tuple(range(token0, token0 + count)))
          for _, token0, row0, count, early, kept in pieces if kept}
    assert on == {(at * page + b * block, early, tuple(tokens))
                  for at, b, early, tokens in ref.blocks_of(off, kv, table, page, block, n, n_pages)}


LEADS = [([20, 21], [1], 16, 16), ([16, 17], [1], 16, 16), ([48, 112], [64], 64, 16), ([300, 301], [1], 64, 16),
         ([300, 300, 420, 421], [0, 177, 9], 128, 32), ([15, 16], [1], 16, 16), ([0, 1], [1], 16, 16)]


@pytest.mark.parametrize("per", [1, 2])
@pytest.mark.parametrize("off,kv,page,block", LEADS)
def test_tokens_before_the_first_sequence(program, off, kv, page, block, per):
    """Tiles of tokens that belong to no sequence take nothing, however many."""
    table = np.arange(len(kv) * 8).reshape(len(kv), 8)[::-1]
    batch = (per, block, page, off[-1] + 5, off, kv, table, table.size)
    check(batch, walk(program, [batch])[0])


def test_random_batches(program):
    rng = np.random.default_rng(401)
    batches = []
    for _ in range(3000):
        n_seqs, page = int(rng.integers(1, 7)), int(rng.choice([16, 64, 256]))
        block = int(rng.choice([b for b in (16, 32, 256) if b <= page]))
        new = rng.integers(0, 120, n_seqs) * (rng.random(n_seqs) < 0.8)
        off = np.concatenate([[0], np.cumsum(new)]) + int(rng.choice([0, rng.integers(0, 400)]))
        kv = new + rng.integers(-20, 300, n_seqs)
        n = max(int(off[-1]) + int(rng.choice([0, 9, -7])), 1)
        width = int(rng.integers(1, 420 // page + 2))
        n_pages = n_seqs * width + 3
        batches.append((int(rng.integers(1, 3)), block, page, n, off, kv,
                        table_of(rng, n_seqs, width, n_pages), n_pages))
    for batch, pieces in zip(batches, walk(program, batches)):
        check(batch, pieces)


def test_any_arrays_stay_within_the_tensors(program):
    """Offsets that fall, and numbers at the ends of 32 bits: pieces of tokens that
    are there, in a block of the pool."""
    rng = np.random.default_rng(402)
    batches = []
    for _ in range(3000):
        n_seqs, n = int(rng.integers(1, 6)), int(rng.integers(1, 300))

        def numbers(k):
            return np.where(rng.random(k) < 0.2, rng.choice([-INT32, INT32 - 1, -1, 0], k),
                            rng.integers(-50, 350, k))
        batches.append((int(rng.integers(1, 3)), 16, 64, n, numbers(n_seqs + 1), numbers(n_seqs),
                        numbers(n_seqs * 3).reshape(n_seqs, 3), 40))
    for (_, block, page, n, *_, n_pages), pieces in zip(batches, walk(program, batches)):
        for _, token0, row0, count, early, _ in pieces:
            assert count > 0 and early >= 0 and early + count <= block
            assert 0 <= token0 and token0 + count <= n
            assert 0 <= row0 and row0 + block <= n_pages * page and row0 % block == 0
