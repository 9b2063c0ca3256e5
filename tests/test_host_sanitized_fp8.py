"""Host code of the block-scaled 8-bit products under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): tests/host/fp8_driver.cpp links
gg_fp8_api.cpp against the fake HIP runtime and its own recording launchers.  A
sanitizer report makes the driver exit non-zero, and so does a failed check."""
import os

import pytest

from test_host_sanitized import HOST, ROOT, _build_and_run


def test_fp8_host_code_under_sanitizers():
    csrc = os.path.join(ROOT, "moe_expert_grouped_ragged_amd", "csrc")
    if not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("HIP headers not installed")
    out = _build_and_run([os.path.join(csrc, "gg_fp8_api.cpp"), os.path.join(HOST, "fake_hip.cpp"),
                          os.path.join(HOST, "fp8_driver.cpp")],
                         ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                          "-I" + csrc, "-I" + HOST], "fp8_driver")
    print(out)
