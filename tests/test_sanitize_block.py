"""AddressSanitizer and UndefinedBehaviorSanitizer run of the router's and the
norm's entry points (api_block.cpp) on the CPU: built with g++, kernel
launchers replaced by host stubs, and run under tests/test_abi_block.py in a
child process with the ASan runtime preloaded."""
import os
import subprocess
import sys

from test_sanitize import ROOT, SAN, _asan_runtime, _run


def test_block_entry_points_under_sanitizers(tmp_path):
    asan = _asan_runtime()
    lib = str(tmp_path / "libmxmoe_block_san.so")
    _run(["g++", "-std=c++17", "-Wall", "-fPIC", "-shared", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
          os.path.join(ROOT, "mxfp8_block_scaled_04_amd", "csrc", "api_block.cpp"),
          os.path.join(ROOT, "tests", "sanitize", "launch_stubs_block.cpp"), "-o", lib])
    env = dict(os.environ, LD_PRELOAD=asan, MXMOE_BLOCK_LIB=lib,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                        "tests/test_abi_block.py"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    log = r.stdout[-4000:] + "\n" + r.stderr[-4000:]
    assert r.returncode == 0, log
    for marker in ("ERROR: AddressSanitizer", "runtime error:", "ERROR: LeakSanitizer"):
        assert marker not in r.stdout + r.stderr, log
    assert " passed" in r.stdout, log
