"""Words of a plan that is none: the tiles of the adapters' products on the CPU, by the
function that their kernels call."""
import os
import subprocess

import test_serve_offsets as base

pytestmark = base.pytestmark


def test_tiles_stay_inside_the_plan(tmp_path):
    exe = str(tmp_path / "adapter_tile")
    cmd = [base.CXX, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__=1",
           "-I", os.path.join(base.ROCM, "include"), "-I", os.path.join(base.REPO, "include"),
           "-I", os.path.join(base.REPO, "w4_gemm_gated_amd", "csrc"),
           os.path.join(base.REPO, "tests", "adapter_tile_driver.cpp"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and "all checks passed" in res.stdout, res.stdout + res.stderr
