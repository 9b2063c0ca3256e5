"""The C boundary's choice of sums on the CPU: unknown ones are refused before any HIP call, also without rows, and
the launches get what the caller or the default chose (tests/host/fp8_sums_driver.cpp, under sanitizers)."""
import os

import pytest

from test_host_sanitized import HOST, ROOT, _build_and_run

P, BIG = 1 << 20, 1 << 28


def test_unknown_sums_are_refused():
    import moe_expert_grouped_ragged_amd as gg
    L = gg.lib
    calls = (lambda m, s: L.gg_fp8_forward_sums(P, 2 * P, m, 4 * P, 2, 48, 64, 1, -1, None, 32 * P, BIG, 600 * P, s, None),
             lambda m, s: L.gg_fp8_dgrad_sums(P, None, 2 * P, m, 4 * P, 2, 48, 64, 2, -1, None, 32 * P, BIG, 600 * P, s, None),
             lambda m, s: L.gg_fp8_glu_forward_sums(P, 2 * P, m, 4 * P, 8 * P, 2, 64, 40, 0, 32 * P, BIG, None, 600 * P, s, None),
             lambda m, s: L.gg_fp8_glu_dgrad_sums(P, 700 * P, 2 * P, m, 4 * P, 8 * P, 2, 64, 40, 0, 32 * P, BIG, 600 * P, s, None))
    for call in calls:
        for bad in (-1, 3, 1 << 30):
            assert call(16, bad) == gg.GG_ERR_INVALID_ARGUMENT and call(0, bad) == gg.GG_ERR_INVALID_ARGUMENT
        for good in gg.FP8_SUMS.values():
            assert call(0, good) == gg.GG_OK


def test_fp8_sums_host_code_under_sanitizers():
    csrc = os.path.join(ROOT, "moe_expert_grouped_ragged_amd", "csrc")
    if not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("HIP headers not installed")
    print(_build_and_run([os.path.join(csrc, "gg_fp8_api.cpp"), os.path.join(HOST, "fake_hip.cpp"),
                          os.path.join(HOST, "fp8_sums_driver.cpp")],
                         ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                          "-I" + csrc, "-I" + HOST], "fp8_sums_driver"))
