"""The attention kernels' loads to LDS, in the assembly that the compiler makes of them: each
leaves the execution mask as it found it, whatever branch it ends up in, and no lambda of a kernel
has become a call or keeps its captures in memory that flat instructions reach."""

import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_sampling_verification_amd", "csrc")


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    hipcc = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not found")
    out = str(tmp_path_factory.mktemp("asm") / "attn.s")
    cmd = [hipcc, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature",
           "-Xclang", "-packed-fp32-ops", "-Wno-unused-command-line-argument", "--cuda-device-only",
           "-S", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(CSRC, "sv_tree_attn.hip"), "-o", out]
    build = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert build.returncode == 0, build.stderr[-4000:]
    with open(out) as f:
        return f.read()


@pytest.mark.timeout(700)
def test_loads_to_lds_keep_the_execution_mask(assembly):
    blocks = re.findall(r";#ASMSTART\n(.*?);;#ASMEND", assembly, re.S)
    loads = [b for b in blocks if "global_load_lds" in b]
    assert len(loads) > 100
    for b in loads:
        lines = [x.strip() for x in b.strip().splitlines()]
        at = next(i for i, x in enumerate(lines) if "global_load_lds" in x)
        assert lines[0].startswith("s_mov_b32 m0,") and at == 2  # a wait state behind m0
        writes = [x for x in lines if re.search(r"\bexec\b", x)]
        if not writes:
            continue
        save = re.match(r"s_and_saveexec_b64 (s\[\d+:\d+\]), s\[\d+:\d+\]$", lines[1])
        assert save and lines[at + 1:] == [f"s_mov_b64 exec, {save.group(1)}"], b


@pytest.mark.timeout(700)
def test_kernels_call_nothing(assembly):
    code = "\n".join(x for x in assembly.splitlines() if not x.lstrip().startswith((".", ";")))
    assert len(re.findall(r"^_ZN.*k_tree_attn.*:", code, re.M)) >= 20
    assert not re.search(r"\b(s_swappc|s_call|flat_(load|store|atomic))", code)
