"""Checks on the machine code of the experts' products (CPU only: the kernels are
compiled to gfx950 assembly here, nothing runs on a GPU).

The weight gradient issues its MFMAs as inline assembly, whose operands the
compiler's hazard logic does not see, and both kernels read their accumulators by
inline assembly behind a fixed wait.  Required of the built code: no VALU write
closer than MIN_WAIT_STATES before an MFMA that reads the register (inline MFMAs
only: the compiler pads its own), no accumulator read closer than a finished MFMA's
wait states, and no scratch traffic in any instance."""
import os
import subprocess
import tempfile

import pytest

from tests.test_kernel_hazards import HIPCC, MIN_WAIT_STATES, ROOT, functions, mfma_hazards

SOURCES = {"gemm_experts_wgrad": "wgrad_kernel", "gemm_experts": "gemm_experts_tile_kernel"}
RESULT_WAIT_STATES = 18  # 16-pass MFMA write, then VALU read


@pytest.fixture(scope="module", params=sorted(SOURCES))
def kernels(request):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "k.s")
        src = os.path.join(ROOT, "tile_scheduling_persistent_amd", "csrc", request.param + ".hip")
        cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               f"-I{os.path.join(ROOT, 'include')}", "-S", "--cuda-device-only", src, "-o", out]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        return request.param, functions(open(out).read(), SOURCES[request.param])


def reads_too_early(ins):
    """Accumulator reads with fewer than RESULT_WAIT_STATES between them and the last
    MFMA before them (straight-line code; s_nop N counts N + 1)."""
    found, since = [], RESULT_WAIT_STATES
    for q in ins:
        if q.startswith("v_mfma"):
            since = 0
        elif q.startswith("v_accvgpr_read") and since < RESULT_WAIT_STATES:
            found.append(q)
        else:
            since += int(q.split()[1]) + 1 if q.startswith("s_nop") else 1
    return found


def test_operands_results_and_spills(kernels):
    name, fns = kernels
    assert len(fns) >= 6, sorted(fns)
    for fn, ins in fns.items():
        nmf, found = mfma_hazards(ins, MIN_WAIT_STATES)
        assert nmf >= 16, fn
        if name == "gemm_experts_wgrad":
            assert not found, (fn, found[:3])
        assert not reads_too_early(ins), (fn, reads_too_early(ins)[:3])
        assert not [q for q in ins if q.startswith("scratch_")], fn


def test_early_reads_are_found():
    ins = ["v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]", "s_nop 7", "v_accvgpr_read_b32 v0, a0"]
    assert reads_too_early(ins) == [ins[2]]
    assert reads_too_early(ins[:1] + ["s_nop 7"] * 3 + ins[2:]) == []
