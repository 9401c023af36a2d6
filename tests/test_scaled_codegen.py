"""Code-generation guards for the kernels of the block-scaled cache and of the pages
of a step (CPU: hipcc cross-compiles gfx950, no GPU needed): scratch memory,
waves a SIMD, and no packed fp32 instructions."""
import concurrent.futures as cf
import os
import re

import pytest

from codegen_util import saved_before_restore
from test_tokens_codegen import HIPCC, _compile

# attend<DT, e4m3 with scales of blocks, DP, EXACT>: most scratch (bytes a lane), by (DP, EXACT)
SCRATCH = {(128, True): 16, (128, False): 16, (256, True): 32, (256, False): 64}


@pytest.fixture(scope="module")
def codegen(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("codegen")
    names = ("append_scaled", "assign", "attention_scaled")
    with cf.ThreadPoolExecutor(3) as ex:
        got = ex.map(lambda n: _compile(f"{n}_kernels.hip", out / f"{n}.s"), names)
    return dict(zip(names, got))


def test_append_kernels(codegen):
    """Blocks of one strip hold four waves a SIMD, which they are dealt out for,
    without scratch; those of two and four strips spill a little, some."""
    _, usage = codegen["append_scaled"]
    heads = {k: u for k, u in usage.items() if "append_heads" in k}
    blocks = {k: u for k, u in usage.items() if "append_blocks" in k}
    assert len(heads) == 20 and len(blocks) == 32
    for k, u in heads.items():
        assert u["ScratchSize"] == 0 and u["Occupancy"] >= 3, f"{k}: {u}"
    for k, u in blocks.items():
        strips = int(re.search(r"ELi(\d)EEE", k).group(1))
        assert u["ScratchSize"] <= {1: 0, 2: 96, 4: 512}[strips] and u["Occupancy"] >= 4, f"{k}: {u}"


def test_assign_kernels(codegen):
    _, usage = codegen["assign"]
    assert len(usage) == 3
    for k, u in usage.items():
        assert u["ScratchSize"] == 0 and u["Occupancy"] >= 4, f"{k}: {u}"


def test_attention_kernels(codegen):
    _, usage = codegen["attention_scaled"]
    seen = 0
    for k, u in usage.items():
        m = re.search(r"attendILi(\d)ELi4ELi(\d+)ELb(\d)EE", k)
        if not m:
            assert u["ScratchSize"] == 0, f"{k}: {u}"
            continue
        seen += 1
        dim = int(m.group(2))
        most = SCRATCH.get((dim, m.group(3) == "1"), 0)
        assert u["ScratchSize"] <= most and u["Occupancy"] >= (1 if dim > 128 else 2), f"{k}: {u}"
    assert seen == 16


@pytest.mark.parametrize("name", ["append_scaled", "assign", "attention_scaled"])
def test_no_packed_fp32(codegen, name):
    asm, _ = codegen[name]
    assert not re.search(r"v_pk_(add|mul|fma)_f32", asm)


def test_append_keeps_its_registers(codegen):
    """No append spills: one whose angles were spilled lost them for lanes that a
    missing weight had switched off."""
    _, usage = codegen["append_scaled"]
    assert len(usage) == 52
    for k, u in usage.items():
        assert u["ScratchSize"] == 0, f"{k}: {u}"


@pytest.mark.parametrize("name", ["append_scaled", "assign", "attention_scaled"])
def test_saves_have_all_lanes(codegen, name):
    assert saved_before_restore(codegen[name][0]) == []
