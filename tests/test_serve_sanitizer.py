"""The serving operators' host code under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only), built as test_host_sanitizer.py builds the
linear layer's: its compiler flags and object cache are used here too."""
import concurrent.futures
import os
import subprocess

import pytest

import test_host_sanitizer as base

SOURCES = ["serve_api.cpp", "kv_cache.hip", "paged_attn.hip", "paged_attn_tile.hip", "verify.hip"]

pytestmark = base.pytestmark


def _headers():
    return base._headers() + [os.path.join(base.INCLUDE, "spear_serve.h")]


def test_serving_host_code_is_clean_under_sanitizers(monkeypatch):
    monkeypatch.setattr(base, "_headers", lambda h=_headers(): h)
    os.makedirs(base.OUT, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(min(len(SOURCES), os.cpu_count() or 2)) as ex:
        objs = list(ex.map(base._object, SOURCES))
    drv = os.path.join(base.OUT, "serve_driver.o")
    base._run([base.CLANGXX, *base.HOST_FLAGS, "-std=c++17", "-I", base.INCLUDE, "-c",
               os.path.join(base.TESTS, "serve_sanitizer_driver.cpp"), "-o", drv])
    exe = os.path.join(base.OUT, "serve_sanitizer_driver")
    base._run([base.CLANGXX, *base.HOST_FLAGS, drv, *objs, "-L", os.path.join(base.ROCM, "lib"), "-lamdhip64",
               f"-Wl,-rpath,{os.path.join(base.ROCM, 'lib')}", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-6000:]
    assert "all checks passed" in out
