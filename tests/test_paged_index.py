"""The paged cache's index arithmetic (fp8_kv_cache_amd/csrc/kv_internal.h),
compiled for the host from the header the kernels are built from and run
under AddressSanitizer and UBSan over random and hostile batches (no GPU)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tiles_tokens_and_pages(tmp_path):
    exe = tmp_path / "paged_index_check"
    cmd = ["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "fp8_kv_cache_amd", "csrc"),
           os.path.join(ROOT, "tests", "paged_index_check.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode and ("hip_runtime" in r.stderr or "cannot find -lasan" in r.stderr):
        pytest.skip("HIP headers or the sanitizer are not usable from g++ here: " + r.stderr[:200])
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:verify_asan_link_order=0"))
    assert out.returncode == 0 and out.stdout.startswith("ok "), out.stdout[-2000:] + out.stderr[-3000:]
