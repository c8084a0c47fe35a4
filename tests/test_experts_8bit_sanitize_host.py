"""The 8-bit expert path's host checks under AddressSanitizer and
UndefinedBehaviorSanitizer (no GPU): moe_experts_8bit_api.cpp and the quantising
permute of moe_permute_api.cpp against the stub HIP runtime and stub launch
layers of tests/sanitize/, driven by the ABI and binding checks in a child
pytest.
"""

import os
import subprocess
import sys

import pytest

from test_sanitize_host import CSRC, FLAGS, ROOT, SAN, _asan_runtime, _gpu_visible

pytestmark = [
    pytest.mark.skipif(_gpu_visible(), reason="the fake-pointer ABI checks run only on a host without a GPU"),
    pytest.mark.skipif(_asan_runtime() is None, reason="gcc with the AddressSanitizer runtime is not available"),
]


def test_8bit_abi_clean_under_sanitizers(tmp_path):
    lib = str(tmp_path / "libmoe_permute_san.so")
    sources = [os.path.join(CSRC, "moe_permute_api.cpp"), os.path.join(CSRC, "moe_experts_8bit_api.cpp"),
               os.path.join(SAN, "launch_stub.cpp"), os.path.join(SAN, "expert_8bit_launch_stub.cpp")]
    subprocess.run(["g++", "-std=c++17", "-Wall", *FLAGS, "-shared", "-I", os.path.join(SAN, "stub_include"),
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC, *sources, "-o", lib], check=True)
    env = dict(os.environ)
    pre = env.get("LD_PRELOAD", "")
    env["LD_PRELOAD"] = _asan_runtime() + ((":" + pre) if pre else "")
    env["ASAN_OPTIONS"] = "detect_leaks=0:abort_on_error=1:halt_on_error=1"
    env["UBSAN_OPTIONS"] = "print_stacktrace=1:halt_on_error=1"
    env["MOE_TEST_PERMUTE_LIB"] = lib  # tests/conftest.py points the binding at it
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "not gpu", "-p", "no:cacheprovider",
           "tests/test_experts_8bit_host.py", "-k", "not exports"]
    res = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert res.returncode == 0 and " passed" in out, out[-4000:]
