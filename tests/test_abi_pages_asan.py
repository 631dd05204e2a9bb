"""The host side of the third part of the C ABI (csrc/cache_api.cpp) built with
AddressSanitizer, and the ABI tests of tests/test_abi_moe.py run against that
build (no GPU: the kernel launchers are stubs that return an error,
tests/asan/cache_launch_stubs.cpp)."""

import os
import shutil
import subprocess
import sys

import pytest

from tests.test_abi_asan import PKG, ROOT, _libasan

OUT = os.path.join(ROOT, "_build", "asan", "libmxq_pages_asan.so")


def test_pages_abi_tests_pass_under_asan():
    gxx, rt = shutil.which("g++"), _libasan()
    if not gxx or not rt:
        pytest.skip("g++ with libasan is not available")
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    stubs = os.path.join(ROOT, "tests", "asan")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address", "-fno-omit-frame-pointer", "-shared", "-fPIC",
           "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"),
           os.path.join(PKG, "csrc", "api.cpp"), os.path.join(PKG, "csrc", "cache_api.cpp"),
           os.path.join(stubs, "launch_stubs.cpp"), os.path.join(stubs, "cache_launch_stubs.cpp"), "-o", OUT]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    code = (
        "import sys; sys.path.insert(0, %r)\n"
        "from nvfp4_quantization_grouped_amd import _lib\n"
        "_lib.LIB_PATH = %r\n"
        "import pytest\n"
        "sys.exit(pytest.main(['-q', '-p', 'no:cacheprovider', %r]))\n"
    ) % (ROOT, OUT, os.path.join(ROOT, "tests", "test_abi_pages.py"))
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:exitcode=86")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, cwd=ROOT, timeout=600)
    out = r.stdout + r.stderr
    assert "ERROR: AddressSanitizer" not in out, out[-4000:]
    assert r.returncode == 0 and " passed" in out, out[-4000:]
