"""Checks on the machine code of the experts' product for few rows (CPU only: it is
compiled to gfx950 assembly here, nothing runs on a GPU): no instance spills."""
import os
import re
import subprocess

import pytest

from tests.test_kernel_hazards import HIPCC, ROOT, functions


def test_no_instance_spills(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = str(tmp_path / "k.s")
    src = os.path.join(ROOT, "tile_scheduling_persistent_amd", "csrc", "gemm_experts.hip")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                        f"-I{os.path.join(ROOT, 'include')}", "-S", "--cuda-device-only", src, "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    asm = open(out).read()
    fns = functions(asm, "gemm_experts_stream_kernel")
    assert len(fns) == 8, sorted(fns)
    for fn, ins in fns.items():
        assert [q for q in ins if q.startswith("v_mfma")], fn
        assert not [q for q in ins if q.startswith("scratch_")], fn
    for fn in fns:
        facts = re.search(r"\.name:\s+" + fn + r"\n(.*?)\.vgpr_spill_count:\s*(\d+)", asm, re.S)
        assert facts and int(facts.group(2)) == 0, fn
        assert re.search(r"\.sgpr_spill_count:\s*0\n", facts.group(1)), fn
