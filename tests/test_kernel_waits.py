"""Waits in the attention tile kernel's own assembly (compiled here, no GPU).

Its waves copy keys and values from memory straight into LDS, each its share of a
tile that all of them read.  A barrier does not wait for such copies: the wave
that asked for them has to, before the barrier that publishes the tile.  That
barrier is the one after which the next copies are requested, so on no path may a
copy, a barrier and another copy follow each other without a wait for all memory
instructions (s_waitcnt vmcnt(0)) somewhere between.
"""
import os
import re
import shutil
import subprocess

import pytest

from w4_gemm_gated_amd import build

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
NONE, COPYING, PAST_BARRIER = range(3)


def kernels(text):
    """{name: instructions and labels in order} of an assembly file's functions."""
    out = {}
    for m in re.finditer(r"^(_Z\w+):.*?\n(.*?)^\.Lfunc_end", text, re.S | re.M):
        lines = (re.sub(r";.*", "", line).strip() for line in m.group(2).splitlines())
        out[m.group(1)] = [x for x in lines if x and (x.startswith(".LBB") or not x.startswith("."))]
    return out


def unpublished_copies(code):
    """Indexes of copies that are reached with earlier ones past a barrier unwaited."""
    at = {x[:-1]: i for i, x in enumerate(code) if x.endswith(":")}
    todo, seen, bad = [(0, NONE)], set(), set()
    while todo:
        i, state = todo.pop()
        if i >= len(code) or (i, state) in seen:
            continue
        seen.add((i, state))
        x = code[i]
        op = x.split()[0]
        if op.startswith(("buffer_load", "global_load")) and (x.split()[-1] == "lds" or "_lds_" in op):
            if state == PAST_BARRIER:
                bad.add(i)
            state = COPYING
        elif op == "s_barrier" and state == COPYING:
            state = PAST_BARRIER
        elif op == "s_waitcnt" and "vmcnt(0)" in x:
            state = NONE
        assert not op.startswith(("s_setpc", "s_swappc", "s_call")), "a path this test does not follow"
        if op == "s_branch" or op.startswith("s_cbranch"):
            todo.append((at[x.split()[1]], state))
        if op not in ("s_branch", "s_endpgm"):
            todo.append((i + 1, state))
    return bad


def test_the_analysis_tells_the_two_apart():
    loop = [".LBB0_0:", "buffer_load_dwordx4 v1, s[0:3], 0 offen lds", "s_cbranch_scc0 .LBB0_1",
            "s_waitcnt vmcnt(0) lgkmcnt(0)", ".LBB0_1:", "s_waitcnt lgkmcnt(0)", "s_barrier", "s_cbranch_scc1 .LBB0_0",
            "s_endpgm"]
    assert unpublished_copies(loop) == {1}
    assert not unpublished_copies(loop[:5] + ["s_waitcnt vmcnt(0)"] + loop[5:])


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_tile_kernels_wait_for_their_copies(tmp_path):
    out = tmp_path / "tile.s"
    cmd = [HIPCC, *build.COMMON_FLAGS, "--cuda-device-only", "-S", os.path.join(build.CSRC, "paged_attn_tile.hip"),
           "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    copying = 0
    for name, code in kernels(out.read_text()).items():
        copying += any(x.split()[-1] == "lds" for x in code)
        bad = unpublished_copies(code)
        assert not bad, (name, [code[i] for i in sorted(bad)])
    assert copying == 2         # fp16 at both head dimensions; 8-bit tiles pass through registers
