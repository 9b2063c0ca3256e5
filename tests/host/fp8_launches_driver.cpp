// Host-side driver of the launches that the fp8 entry points make: the counts
// that include/gg.h promises, at both sides of each condition.  Built with the
// fake HIP runtime and the counting launchers below, under sanitizers, by
// tests/test_fp8_launches.py.  Exit status 0 when every check holds.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "fake_hip.h"
#include "gg.h"
#include "gg_fp8.h"

static int g_launches;

namespace gg {
hipError_t launch_f8_quant(F8Mode, const F8QuantParams&, int, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_f8_gemm(F8Epilogue, const F8Params&, int, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_f8_quant_weights(const uint16_t*, int, const F8Dim&, const F8Dim&, uint8_t*, uint8_t*, hipStream_t) { return hipSuccess; }
hipError_t launch_f8_pack(const uint8_t*, const uint8_t*, int, const F8Dim&, const F8Dim&, int, uint8_t*, hipStream_t) { return hipSuccess; }
}  // namespace gg

static int g_failed = 0, g_checked = 0;
static void check(const char* what, int64_t M, int64_t E, int64_t width, int status, int want) {
    ++g_checked;
    if (status != GG_OK || g_launches != want) {
        ++g_failed;
        std::fprintf(stderr, "%s, M %lld, E %lld, width %lld: status %d, %d launches, not %d\n", what, static_cast<long long>(M),
                     static_cast<long long>(E), static_cast<long long>(width), status, g_launches, want);
    }
    g_launches = 0;
}

int main() {
    // one allocation in parts that do not overlap; nothing is read from it
    constexpr size_t PART = 64 << 20;
    std::vector<uint8_t> raw(PART * 7 + 64);
    uint8_t* base = raw.data() + ((16 - (reinterpret_cast<uintptr_t>(raw.data()) & 15)) & 15);
    auto part = [&](int i) { return base + i * PART; };
    int64_t* off = reinterpret_cast<int64_t*>(part(6));
    hipStream_t s = fake_stream(0);
    const int none = GG_ACT_NONE, act = GG_ACT_SWIGLU;
    for (int64_t M : {1, 16, 17, 64, 65})
        for (int64_t E : {1, 3, 7, 8})
            for (int64_t K : {64, 4096, 4104}) {
                const int64_t N = 64;
                const int one = M <= 64 && M <= 8 * (E + 1) && (K + 127) / 128 * 128 <= 4096 ? 1 : 2;
                check("forward", M, E, K, gg_fp8_forward(part(0), off, M, part(1), E, N, K, 1, none, nullptr, part(2), PART, part(3), s), one);
                check("forward of A", M, E, K, gg_fp8_forward(part(0), off, M, part(1), E, N, K, 1, act, nullptr, part(2), PART, part(3), s), 2);
                check("gradient", M, E, K, gg_fp8_dgrad(part(0), nullptr, off, M, part(1), E, K, N, 1, none, nullptr, part(2), PART, part(3), s), one);
                check("block", M, E, K, gg_fp8_glu_forward(part(0), off, M, part(1), part(4), E, K, N, act, part(2), PART, nullptr, part(3), s), one + 1);
                check("its gradient", M, E, K, gg_fp8_glu_dgrad(part(0), part(5), off, M, part(1), part(4), E, K, N, act, part(2), PART, part(3), s),
                      one + 1);
                // halves of W1: each in whole blocks
                const int64_t F = K / 2 / 8 * 8, blocks = 2 * ((F + 127) / 128 * 128);
                const int half = M <= 64 && M <= 8 * (E + 1) && blocks <= 4096 ? 1 : 2;
                check("gradient of halves", M, E, 2 * F,
                      gg_fp8_dgrad(part(0), nullptr, off, M, part(1), E, 2 * F, N, 2, none, nullptr, part(2), PART, part(3), s), half);
                check("gradient of dH1", M, E, 2 * F,
                      gg_fp8_dgrad(part(0), part(5), off, M, part(1), E, 2 * F, N, 2, act, nullptr, part(2), PART, part(3), s), 2);
            }
    std::printf("%d of %d checks failed\n", g_failed, g_checked);
    return g_failed ? 1 : 0;
}
