"""The weighing kernels' loads to LDS, in the assembly that the compiler makes of them: they leave the
execution mask alone, with a wait state behind their address, and nothing in a kernel has become a
call or is reached through private memory by flat instructions."""

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
    out = str(tmp_path_factory.mktemp("asm") / "weigh.s")
    cmd = [hipcc, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature",
           "-Xclang", "-packed-fp32-ops", "-Wno-unused-command-line-argument", "--cuda-device-only",
           "-S", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(CSRC, "sv_weigh.hip"), "-o", out]
    build = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert build.returncode == 0, build.stderr[-4000:]
    with open(out) as f:
        return f.read()


@pytest.mark.timeout(700)
def test_loads_to_lds(assembly):
    blocks = re.findall(r";#ASMSTART\n(.*?);;#ASMEND", assembly, re.S)
    loads = [b for b in blocks if "global_load_lds" in b]
    assert len(loads) >= 30
    for b in loads:
        lines = [x.strip() for x in b.strip().splitlines()]
        assert lines[0].startswith("s_mov_b32 m0,") and lines[1] == "s_nop 0"
        assert lines[2].startswith("global_load_lds_dwordx4") and len(lines) == 3
        assert not re.search(r"\bexec\b", b)


@pytest.mark.timeout(700)
def test_kernels_call_nothing(assembly):
    code = "\n".join(x for x in assembly.splitlines() if not x.lstrip().startswith((".", ";")))
    # of both types and four head sizes each
    for name in ("k_weigh", "k_weigh_rows"):
        found = re.findall(rf"^_ZN\w*\d{name}ILb([01])ELi(\d+)E\w*:", code, re.M)
        assert set(found) == {(t, d) for t in "01" for d in ("64", "96", "128", "256")}
    assert not re.search(r"\b(s_swappc|s_call|flat_(load|store|atomic))", code)
