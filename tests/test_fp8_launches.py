"""The numbers of launches that include/gg.h states for the fp8 calls (CPU only; tests/host/fp8_launches_driver.cpp under sanitizers)."""
import os

import pytest

from test_host_sanitized import HOST, ROOT, _build_and_run


def test_launches_are_those_of_the_header():
    csrc = os.path.join(ROOT, "moe_expert_grouped_ragged_amd", "csrc")
    if not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("HIP headers not installed")
    print(_build_and_run([os.path.join(csrc, "gg_fp8_api.cpp"), os.path.join(HOST, "fake_hip.cpp"),
                          os.path.join(HOST, "fp8_launches_driver.cpp")],
                         ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                          "-I" + csrc, "-I" + HOST], "fp8_launches_driver"))
