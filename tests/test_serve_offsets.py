"""Offsets that do not rise from zero: the read-back's places on the CPU, by the
function that its kernel calls."""
import os
import shutil
import subprocess

import pytest

REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = "/opt/rocm"
CXX = shutil.which("g++") or os.path.join(ROCM, "llvm", "bin", "clang++")

pytestmark = pytest.mark.skipif(not os.path.exists(CXX) or not os.path.exists(os.path.join(ROCM, "include", "hip")),
                                reason="needs a host compiler and the HIP headers")


def test_read_back_places_stay_inside_the_table(tmp_path):
    exe = str(tmp_path / "kv_place")
    cmd = [CXX, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__=1",
           "-I", os.path.join(ROCM, "include"), "-I", os.path.join(REPO, "include"),
           "-I", os.path.join(REPO, "w4_gemm_gated_amd", "csrc"), os.path.join(REPO, "tests", "kv_place_driver.cpp"),
           "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and "all checks passed" in res.stdout, res.stdout + res.stderr


def test_attention_counts_that_offsets_could_overflow_are_known(tmp_path):
    exe = str(tmp_path / "attn_counts")
    cmd = [CXX, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__=1",
           "-I", os.path.join(ROCM, "include"), "-I", os.path.join(REPO, "include"),
           "-I", os.path.join(REPO, "w4_gemm_gated_amd", "csrc"), os.path.join(REPO, "tests", "attn_counts_driver.cpp"),
           "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and "all checks passed" in res.stdout, res.stdout + res.stderr
