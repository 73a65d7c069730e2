"""The paged-cache entry points' host code (api_paged.cpp) under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU, with the launchers and HIP runtime calls stubbed."""
import os
import shutil

import pytest

from test_sanitizers import ROOT, SAN, _build_and_run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_paged_host_code_under_address_and_undefined_behaviour_sanitizers(tmp_path):
    exe = tmp_path / "paged_asan"
    csrc = os.path.join(ROOT, "quantized_matmul_mlx_amd", "csrc")
    _build_and_run(tmp_path, ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
                              "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                              "-I" + os.path.join(ROOT, "include"), "-I" + csrc, "-o", str(exe),
                              os.path.join(csrc, "api_paged.cpp"), os.path.join(SAN, "paged_driver.cpp")], exe)
