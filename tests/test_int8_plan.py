"""Which kernels the 8-bit products launch, on the CPU: tests/host/int8_plan_driver.cpp
under AddressSanitizer and UndefinedBehaviorSanitizer."""
import os

import pytest

from test_host_sanitized import HOST, ROOT, _build_and_run


def test_launches_of_the_sizes():
    if not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("HIP headers not installed")
    csrc = os.path.join(ROOT, "moe_expert_grouped_ragged_amd", "csrc")
    _build_and_run([os.path.join(HOST, "int8_plan_driver.cpp")],
                   ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + csrc], "int8_plan_driver")
