"""The paged-cache entry points' host code (api_paged.cpp) under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU, with the launchers and HIP runtime calls stubbed."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_paged_host_code_under_address_and_undefined_behaviour_sanitizers(tmp_path):
    exe = tmp_path / "paged_asan"
    csrc = os.path.join(ROOT, "quantized_matmul_mlx_amd", "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                        "-I" + os.path.join(ROOT, "include"), "-I" + csrc, "-o", str(exe),
                        os.path.join(csrc, "api_paged.cpp"), os.path.join(ROOT, "tests", "sanitize", "paged_driver.cpp")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "all checks passed" in out, out
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out
