"""Code-generation guards for the token kernels (CPU: hipcc cross-compiles
gfx950, no GPU needed).

Compiles rope_kernels.hip and attention_kernels.hip with the compiler's
resource-usage remarks and checks:
  * norm, rotation, gradient and append use no scratch memory and keep the waves
    they were measured with (forward and append six a SIMD, gradient three);
  * attention on heads of up to 96 uses no scratch; wider ones, whose rows fill
    the registers, no more than they were measured with (bytes a lane);
  * no packed fp32 instructions.
"""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "depth_weighted_scatter_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"

# attend<DT, CDT, DP, EXACT> (1 fp16, 2 e4m3, 3 bf16): most scratch, by (e4m3, DP, EXACT)
SCRATCH = {(False, 128, True): 16, (False, 128, False): 28, (True, 128, True): 80,
           (True, 128, False): 48, (False, 256, True): 196, (False, 256, False): 412,
           (True, 256, True): 388, (True, 256, False): 428}


def _compile(source, out):
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-S",
           "-Rpass-analysis=kernel-resource-usage", os.path.join(CSRC, source), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-3000:]
    usage, name = {}, None
    for line in r.stderr.splitlines():
        m = re.search(r"Function Name: (\S+)", line)
        if m:
            name = m.group(1)
            usage[name] = {}
        m = re.search(r"remark:.*?\s(ScratchSize \[bytes/lane\]|Occupancy \[waves/SIMD\]): (\d+)", line)
        if m and name:
            usage[name][m.group(1).split()[0]] = int(m.group(2))
    return out.read_text(), usage


@pytest.fixture(scope="module")
def codegen(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("codegen")
    names = ("rope", "attention")
    with cf.ThreadPoolExecutor(2) as ex:
        got = ex.map(lambda n: _compile(f"{n}_kernels.hip", out / f"{n}.s"), names)
    return dict(zip(names, got))


def test_norm_and_append_kernels(codegen):
    _, usage = codegen["rope"]
    for kernel, count, waves in (("norm_rope_fwd", 30, 6), ("norm_rope_bwd", 30, 3), ("6append", 40, 6)):
        found = {k: u for k, u in usage.items() if kernel in k}
        assert len(found) == count
        for k, u in found.items():
            assert u["ScratchSize"] == 0 and u["Occupancy"] >= waves, f"{k}: {u}"


def test_attention_kernels(codegen):
    _, usage = codegen["attention"]
    seen = 0
    for k, u in usage.items():
        m = re.search(r"attendILi(\d)ELi(\d)ELi(\d+)ELb(\d)EE", k)
        if not m:
            assert u["ScratchSize"] == 0, f"{k}: {u}"
            continue
        seen += 1
        dim = int(m.group(3))
        most = SCRATCH.get((m.group(2) == "2", dim, m.group(4) == "1"), 0)
        assert u["ScratchSize"] <= most and u["Occupancy"] >= (1 if dim > 128 else 2), f"{k}: {u}"
    assert seen == 32


@pytest.mark.parametrize("name", ["rope", "attention"])
def test_no_packed_fp32(codegen, name):
    asm, _ = codegen[name]
    assert not re.search(r"v_pk_(add|mul|fma)_f32", asm)
