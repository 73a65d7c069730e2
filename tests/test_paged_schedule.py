"""The launches of paged attention (paged_sched.h, plain host arithmetic) hold all the work that the
kernels find in a call: counted request by request on the CPU, under AddressSanitizer and
UndefinedBehaviorSanitizer."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_launches_hold_the_work_of_every_call(tmp_path):
    exe = tmp_path / "paged_sched"
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                        "-I" + os.path.join(ROOT, "quantized_matmul_mlx_amd", "csrc"), "-o", str(exe),
                        os.path.join(ROOT, "tests", "sanitize", "paged_sched_driver.cpp")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "all checks passed" in out, out
