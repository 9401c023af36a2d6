"""Whether a step of pages can be carried out: the sums its kernel decides by, compiled
for the host, against whole numbers of any size (CPU, no GPU needed)."""
import os
import subprocess

import numpy as np
import pytest

from test_tokens_codegen import CSRC, HIPCC, ROOT

MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("plan") / "plan")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", f"-I{os.path.join(ROOT, 'include')}",
           f"-I{CSRC}", os.path.join(ROOT, "tests", "assign_plan_main.hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]

    def run(steps):
        words = [w for s in steps for w in (*s[:5], len(s[5]), *(x for seq in s[5] for x in seq))]
        r = subprocess.run([out], input=" ".join(map(str, words)), capture_output=True, text=True, timeout=60)
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return run


def expected(n_tokens, n_free, listed, shift, max_pages, seqs):
    count, room, page = min(max(listed, 0), n_free), max_pages << shift, 1 << shift
    tokens = taken = returned = 0
    fits = True
    for kv, keep, new in seqs:
        kv, new = max(kv, 0), max(new, 0)
        keep = min(max(keep, 0), kv)
        fits &= kv <= room and keep + new <= room
        more = -(-(keep + new) // page) - -(-kv // page)
        tokens, taken, returned = tokens + new, taken + max(more, 0), returned + max(-more, 0)
    left = count + returned - taken
    if not fits or tokens > n_tokens or left > n_free:
        return -1, 0, 0
    return (-left, 0, 0) if left < 0 else (0, taken, returned)


# n_tokens, list, filled, page shift, pages a sequence, (kv, keep, new) of each
FAR = [
    # past 2^31 tokens, with pages for all of them, where n_tokens itself is the largest there is
    (MOST, 2 ** 24, 2 ** 24, 8, 2 ** 22, [(0, 0, 2 ** 30)] * 3),
    (MOST, 2 ** 24, 2 ** 24, 8, 2 ** 22, [(0, 0, 2 ** 30)] * 5),
    (MOST, 2 ** 24, 2 ** 24, 8, 2 ** 22, [(0, 0, 2 ** 30), (0, 0, 2 ** 30)]),
    (MOST, 2 ** 24, 2 ** 24, 8, 2 ** 22, [(0, 0, 2 ** 30), (0, 0, 2 ** 30 - 1)]),
    (MOST - 1, 2 ** 24, 2 ** 24, 8, 2 ** 22, [(0, 0, 2 ** 30), (0, 0, 2 ** 30 - 1)]),
    # tokens that need no page, in places on pages that are there
    (MOST, 16, 0, 8, 1, [(1, 1, 255)] * 9000000),
]


@pytest.mark.parametrize("step", FAR, ids=range(len(FAR)))
def test_tokens_past_32_bits(plan, step):
    assert plan([step])[0][:3] == expected(*step)


def test_random_steps(plan):
    rng = np.random.default_rng(404)
    steps = []
    for _ in range(3000):
        shift, width = int(rng.integers(4, 9)), int(rng.integers(0, 12))

        def number(most):
            return int(rng.choice([rng.integers(-3, most + 2), rng.integers(0, most + 1), -2 ** 31, MOST],
                                  p=[0.3, 0.66, 0.02, 0.02]))
        room = max(width << shift, 1)
        seqs = [(number(room), number(room), number(room // 2)) for _ in range(int(rng.integers(0, 7)))]
        n_free = int(rng.integers(0, 40))
        steps.append((int(rng.integers(0, 4 * room)), n_free, int(rng.integers(-2, n_free + 3)), shift, width, seqs))
    got = plan(steps)
    assert [g[:3] for g in got] == [expected(*s) for s in steps]
    assert len({g[0] > 0 for g in got}) == 2 and any(g[0] == 0 for g in got)
