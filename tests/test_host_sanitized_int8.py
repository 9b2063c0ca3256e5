"""Host code of the 8-bit products and the adapters under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): tests/host/int8_adapter_driver.cpp links
gg_int8_api.cpp and gg_adapter_api.cpp against the fake HIP runtime and its own
recording launchers.  A sanitizer report makes the driver exit non-zero, and so
does a failed check."""
import os

import pytest

from test_host_sanitized import HOST, ROOT, _build_and_run


def test_int8_and_adapter_host_code_under_sanitizers():
    csrc = os.path.join(ROOT, "moe_expert_grouped_ragged_amd", "csrc")
    if not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("HIP headers not installed")
    out = _build_and_run([os.path.join(csrc, "gg_int8_api.cpp"), os.path.join(csrc, "gg_adapter_api.cpp"),
                          os.path.join(HOST, "fake_hip.cpp"), os.path.join(HOST, "int8_adapter_driver.cpp")],
                         ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                          "-I" + csrc, "-I" + HOST], "int8_adapter_driver")
    print(out)
