// Host-side driver of the choice of sums in gg_fp8_api.cpp: which products of
// each entry point sum in fp32, by default and as asked for.  Built with the
// fake HIP runtime and the recording launchers below, under sanitizers, by
// tests/test_fp8_sums_boundary.py.  Exit status 0 when every check holds.
#include <cstdint>
#include <cstdio>
#include <string>
#include <vector>

#include "fake_hip.h"
#include "gg.h"
#include "gg_fp8.h"

static std::string g_sums;   // a digit for each product: its fp32_sums

namespace gg {
hipError_t launch_f8_quant(F8Mode, const F8QuantParams&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_f8_gemm(F8Epilogue, const F8Params& p, int, hipStream_t) {
    g_sums += static_cast<char>('0' + p.fp32_sums);
    return hipSuccess;
}
hipError_t launch_f8_quant_weights(const uint16_t*, int, const F8Dim&, const F8Dim&, uint8_t*, uint8_t*, hipStream_t) { return hipSuccess; }
hipError_t launch_f8_pack(const uint8_t*, const uint8_t*, int, const F8Dim&, const F8Dim&, int, uint8_t*, hipStream_t) { return hipSuccess; }
}  // namespace gg

static int g_failed = 0, g_checked = 0;
static void check(const char* what, int status, const char* want) {
    ++g_checked;
    if (status != GG_OK || g_sums != want) {
        ++g_failed;
        std::fprintf(stderr, "%s: status %d, sums %s, not %s\n", what, status, g_sums.c_str(), want);
    }
    g_sums.clear();
}

int main() {
    const int64_t E = 2, H = 64, F = 64, M = 100;
    std::vector<uint8_t> raw(8 << 20);
    uint8_t* at = raw.data() + ((16 - (reinterpret_cast<uintptr_t>(raw.data()) & 15)) & 15);
    auto take = [&](size_t n) {
        uint8_t* p = at;
        at += (n + 15) / 16 * 16;
        return p;
    };
    const size_t need = gg_fp8_glu_workspace_bytes(M, H, F, 1);
    uint8_t *x = take(M * 2 * F * 2), *h1 = take(M * 2 * F * 2), *y = take(M * 2 * F * 2), *ws = take(need), *w = take(gg_fp8_packed_bytes(E, 2 * F, H, 2)),
            *v = take(gg_fp8_packed_bytes(E, 2 * F, H, 2));
    int64_t* off = reinterpret_cast<int64_t*>(take((E + 1) * 8));
    off[E] = M;
    hipStream_t s = fake_stream(0);
    const int none = GG_ACT_NONE, act = GG_ACT_SWIGLU;
    const struct { int sums; const char *single, *w1, *block; } want[] = {
        {GG_FP8_SUMS_DEFAULT, "0", "1", "10"}, {GG_FP8_SUMS_FP32, "1", "1", "11"}, {GG_FP8_SUMS_SCALED, "0", "0", "00"}};
    for (const auto& t : want) {
        // y: of x, or of A; H1; dx: of dY, or behind the derivative; dA
        check("y", gg_fp8_forward_sums(x, off, M, w, E, H, F, 1, none, nullptr, ws, need, y, t.sums, s), t.single);
        check("y of A", gg_fp8_forward_sums(h1, off, M, w, E, H, F, 1, act, nullptr, ws, need, y, t.sums, s), t.single);
        check("H1", gg_fp8_forward_sums(x, off, M, w, E, 2 * F, H, 2, none, nullptr, ws, need, y, t.sums, s), t.w1);
        check("dx", gg_fp8_dgrad_sums(x, nullptr, off, M, w, E, 2 * F, H, 2, none, nullptr, ws, need, y, t.sums, s), t.single);
        check("dx of dH1", gg_fp8_dgrad_sums(x, h1, off, M, w, E, 2 * F, H, 2, act, nullptr, ws, need, y, t.sums, s), t.single);
        check("dA", gg_fp8_dgrad_sums(x, nullptr, off, M, w, E, H, F, 1, none, nullptr, ws, need, y, t.sums, s), t.w1);
        check("block", gg_fp8_glu_forward_sums(x, off, M, w, v, E, H, F, act, ws, need, nullptr, y, t.sums, s), t.block);
        check("block's gradient", gg_fp8_glu_dgrad_sums(x, h1, off, M, w, v, E, H, F, act, ws, need, y, t.sums, s), t.block);
    }
    check("plain y", gg_fp8_forward(x, off, M, w, E, H, F, 1, none, nullptr, ws, need, y, s), "0");
    check("plain H1", gg_fp8_forward(x, off, M, w, E, 2 * F, H, 2, none, nullptr, ws, need, y, s), "1");
    check("plain dx", gg_fp8_dgrad(x, nullptr, off, M, w, E, 2 * F, H, 2, none, nullptr, ws, need, y, s), "0");
    check("plain dA", gg_fp8_dgrad(x, nullptr, off, M, w, E, H, F, 1, none, nullptr, ws, need, y, s), "1");
    check("plain block", gg_fp8_glu_forward(x, off, M, w, v, E, H, F, act, ws, need, nullptr, y, s), "10");
    check("plain gradient", gg_fp8_glu_dgrad(x, h1, off, M, w, v, E, H, F, act, ws, need, y, s), "10");
    std::printf("%d of %d checks failed\n", g_failed, g_checked);
    return g_failed ? 1 : 0;
}
