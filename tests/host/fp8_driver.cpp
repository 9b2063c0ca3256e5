// Host-side driver of the C-ABI layer of the block-scaled 8-bit products
// (gg_fp8_api.cpp) built with the fake HIP runtime and the recording launchers
// below: the launches each entry point makes and their parameters, the
// workspace's layout, sizes at the largest allowed counts, device checks,
// runtime errors and the debug offset check.  Built and run under
// AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_host_sanitized_fp8.py.  Exit status 0 when every check holds.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "fake_hip.h"
#include "gg.h"
#include "gg_fp8.h"

namespace {

struct Record {
    int kind;   // 0 quantize, 1 multiply, 2 quantize weights, 3 pack
    gg::F8Mode mode;
    gg::F8Epilogue epilogue;
    gg::F8QuantParams q;
    gg::F8Params g;
    int num_cu;
    hipStream_t stream;
};
std::vector<Record> g_rec;
int g_fail_kind = -1;

hipError_t result(int kind) { return kind == g_fail_kind ? hipErrorLaunchFailure : hipSuccess; }

}  // namespace

namespace gg {
hipError_t launch_f8_quant(F8Mode mode, const F8QuantParams& p, int num_cu, hipStream_t s) {
    Record r{};
    r.kind = 0, r.mode = mode, r.q = p, r.num_cu = num_cu, r.stream = s;
    g_rec.push_back(r);
    return result(0);
}
hipError_t launch_f8_gemm(F8Epilogue epilogue, const F8Params& p, int num_cu, hipStream_t s) {
    Record r{};
    r.kind = 1, r.epilogue = epilogue, r.g = p, r.num_cu = num_cu, r.stream = s;
    g_rec.push_back(r);
    return result(1);
}
hipError_t launch_f8_quant_weights(const uint16_t*, int, const F8Dim&, const F8Dim&, uint8_t*, uint8_t*, hipStream_t) {
    Record r{};
    r.kind = 2;
    g_rec.push_back(r);
    return result(2);
}
hipError_t launch_f8_pack(const uint8_t*, const uint8_t*, int, const F8Dim&, const F8Dim&, int, uint8_t*, hipStream_t) {
    Record r{};
    r.kind = 3;
    g_rec.push_back(r);
    return result(3);
}
}  // namespace gg

static int g_failed = 0, g_checked = 0;
#define CHECK(cond)                                                              \
    do {                                                                         \
        ++g_checked;                                                             \
        if (!(cond)) {                                                           \
            ++g_failed;                                                          \
            std::fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
        }                                                                        \
    } while (0)

// 16-byte aligned host buffers standing in for device memory.
struct Buf {
    std::vector<uint8_t> raw;
    uint8_t* p;
    explicit Buf(size_t n) : raw(n + 64, 0) {
        p = raw.data() + ((16 - (reinterpret_cast<uintptr_t>(raw.data()) & 15)) & 15);
    }
    template <typename T> T* as() { return reinterpret_cast<T*>(p); }
};

static void test_products() {
    const int64_t E = 3, N = 304, K = 264, M = 100;
    Buf x(M * 2 * K * 2), off((E + 1) * 8), w(gg_fp8_packed_bytes(E, N, K, 2)), a(M * K * 2), y(M * N * 2);
    const size_t need = gg_fp8_workspace_bytes(M, K, 1);
    Buf ws(need);
    off.as<int64_t>()[E] = M;
    hipStream_t s = fake_stream(0);
    g_rec.clear();
    CHECK(gg_fp8_forward(x.p, off.as<int64_t>(), M, w.p, E, N, K, 2, GG_ACT_QGEGLU, a.p, ws.p, need, y.p, s) == GG_OK);
    CHECK(g_rec.size() == 2 && g_rec[0].kind == 0 && g_rec[1].kind == 1 && g_rec[0].stream == s && g_rec[1].stream == s);
    const gg::F8QuantParams q = g_rec[0].q;
    CHECK(g_rec[0].mode == gg::F8_GLU && q.slope == 1.702f && q.dim.real() == K && q.dim.padded() == 384 && q.M == M);
    CHECK(q.q == ws.p && q.s == ws.p + M * 384 && q.s + M * 4 == ws.p + need && q.v_out == a.as<uint16_t>());
    const gg::F8Params g = g_rec[1].g;
    CHECK(g_rec[1].epilogue == gg::F8_STORE && g.q == q.q && g.s == q.s && g.kblocks == 3 && !g.x && g_rec[1].num_cu == 256);
    CHECK(g.n.parts == 2 && g.n.part == 152 && g.n.part_p == 256 && g.n.real() == N && g.n.blocks() == 4);
    CHECK(g.w_stride == 512 * 384 && g.ws == w.p + E * g.w_stride && g.ws_ld == 4 && g.ws_stride == 16);
    CHECK(static_cast<size_t>(g.ws + E * g.ws_stride - w.p) <= gg_fp8_packed_bytes(E, N, K, 2));
    // the gradient: the summed dimension has the halves
    Buf h1(M * N * 2), dh(M * N * 2), dx(M * K * 2), ws2(gg_fp8_workspace_bytes(M, N, 2));
    g_rec.clear();
    CHECK(gg_fp8_dgrad(y.p, h1.p, off.as<int64_t>(), M, w.p, E, N, K, 2, GG_ACT_SWIGLU, dh.p, ws2.p,
                       gg_fp8_workspace_bytes(M, N, 2), dx.p, s) == GG_OK);
    CHECK(g_rec.size() == 2 && g_rec[0].mode == gg::F8_DGLU && g_rec[0].q.h1 == h1.as<uint16_t>());
    CHECK(g_rec[0].q.dim.parts == 2 && g_rec[0].q.dim.part_p == 256 && g_rec[1].g.kblocks == 4);
    CHECK(g_rec[1].g.n.real() == K && g_rec[1].g.ws_stride == 3 * 4);
    // few rows: the product quantizes them; a wide sum, or an expert of many of them: a launch does
    g_rec.clear();
    CHECK(gg_fp8_forward(x.p, off.as<int64_t>(), 32, w.p, E, N, K, 2, GG_ACT_NONE, nullptr, ws.p, need, y.p, s) == GG_OK);
    CHECK(g_rec.size() == 1 && g_rec[0].g.x == x.as<uint16_t>() && g_rec[0].g.k.real() == K);
    CHECK(!gg::f8_quantizes(33, 3, gg::f8_dim(K, 1)) && !gg::f8_quantizes(65, 128, gg::f8_dim(K, 1)));
    CHECK(gg::f8_quantizes(64, 128, gg::f8_dim(4096, 1)) && !gg::f8_quantizes(1, 1, gg::f8_dim(4104, 1)));
    g_rec.clear();
    CHECK(gg_fp8_forward(x.p, off.as<int64_t>(), 8, w.p, E, N, K, 2, GG_ACT_SWIGLU, nullptr, ws.p, need, y.p, s) == GG_OK);
    CHECK(g_rec.size() == 2 && g_rec[0].mode == gg::F8_GLU && !g_rec[0].q.v_out);
    // no rows: success, no launch
    g_rec.clear();
    CHECK(gg_fp8_forward(nullptr, nullptr, 0, nullptr, E, N, K, 1, -1, nullptr, nullptr, 0, nullptr, s) == GG_OK);
    CHECK(g_rec.empty());
    // a launch that fails is an error, and nothing follows it
    for (int kind = 0; kind < 2; ++kind) {
        g_rec.clear();
        g_fail_kind = kind;
        CHECK(gg_fp8_forward(x.p, off.as<int64_t>(), M, w.p, E, N, K, 2, -1, nullptr, ws.p, need, y.p, s) == GG_ERR_HIP);
        CHECK(g_rec.size() == static_cast<size_t>(kind + 1));
    }
    Buf qw(E * N * K), sw(gg_fp8_scale_bytes(E, N, K, 2)), bw(E * N * K * 2);
    g_fail_kind = 2;
    CHECK(gg_fp8_quantize_weights(bw.p, E, N, K, 2, qw.p, sw.p, s) == GG_ERR_HIP);
    g_fail_kind = 3;
    CHECK(gg_fp8_pack(qw.p, sw.p, E, N, K, 2, 1, w.p, gg_fp8_packed_bytes(E, N, K, 2), s) == GG_ERR_HIP);
    g_fail_kind = -1;
    CHECK(gg_fp8_pack(qw.p, sw.p, E, N, K, 2, 1, w.p, gg_fp8_packed_bytes(E, N, K, 2), s) == GG_OK);
}

static void test_block() {
    const int64_t E = 3, H = 136, F = 152, M = 100;
    Buf x(M * H * 2), off((E + 1) * 8), fc1(gg_fp8_packed_bytes(E, 2 * F, H, 2)), fc2(gg_fp8_packed_bytes(E, H, F, 1));
    const size_t need = gg_fp8_glu_workspace_bytes(M, H, F, 0), dneed = gg_fp8_glu_workspace_bytes(M, H, F, 1);
    Buf h1(M * F * 4), y(M * H * 2), ws(need), ws2(dneed);
    off.as<int64_t>()[E] = M;
    hipStream_t s = fake_stream(0);
    g_rec.clear();
    CHECK(gg_fp8_glu_forward(x.p, off.as<int64_t>(), M, fc1.p, fc2.p, E, H, F, GG_ACT_SWIGLU, ws.p, need, h1.p, y.p, s) == GG_OK);
    CHECK(g_rec.size() == 3 && g_rec[0].kind == 0 && g_rec[1].epilogue == gg::F8_STORE_GLU && g_rec[2].epilogue == gg::F8_STORE);
    const gg::F8Params f1 = g_rec[1].g, f2 = g_rec[2].g;
    CHECK(f1.out == h1.as<uint16_t>() && f1.q == ws.p && f1.q_out == f2.q && f1.s_out == f2.s && f1.slope == 1.0f);
    CHECK(f2.q >= f1.s + M * 4 && f2.q - ws.p == M * 260 / 256 * 256 + 256 && f2.s == f2.q + M * 256);
    CHECK(static_cast<size_t>(f2.s + M * 4 - ws.p) <= need);
    CHECK(f1.n.parts == 2 && f1.n.part == F && f1.kblocks == 2 && f2.kblocks == 2 && f2.n.real() == H);
    g_rec.clear();
    CHECK(gg_fp8_glu_forward(x.p, off.as<int64_t>(), 20, fc1.p, fc2.p, E, H, F, GG_ACT_SWIGLU, ws.p, need, nullptr, y.p, s) == GG_OK);
    CHECK(g_rec.size() == 2 && g_rec[0].g.x == x.as<uint16_t>() && !g_rec[0].g.out && !g_rec[1].g.x);
    g_rec.clear();
    CHECK(gg_fp8_glu_dgrad(x.p, h1.p, off.as<int64_t>(), M, fc1.p, fc2.p, E, H, F, GG_ACT_QGEGLU, ws2.p, dneed, y.p, s) == GG_OK);
    CHECK(g_rec.size() == 3 && g_rec[1].epilogue == gg::F8_STORE_DGLU && g_rec[1].g.w == fc2.p && g_rec[2].g.w == fc1.p);
    const gg::F8Params d1 = g_rec[1].g, d2 = g_rec[2].g;
    CHECK(d1.h1 == h1.as<uint16_t>() && d1.slope == 1.702f && d1.n.real() == F && d1.n.parts == 1 && d1.q_out == d2.q);
    CHECK(d2.kblocks == 4 && d2.s == d2.q + M * 512 && static_cast<size_t>(d2.s + M * 4 - ws2.p) <= dneed);
    for (int kind = 0; kind < 2; ++kind) {
        g_rec.clear();
        g_fail_kind = kind;
        CHECK(gg_fp8_glu_dgrad(x.p, h1.p, off.as<int64_t>(), M, fc1.p, fc2.p, E, H, F, 0, ws2.p, dneed, y.p, s) == GG_ERR_HIP);
        CHECK(g_rec.size() == static_cast<size_t>(kind + 1));
    }
    g_fail_kind = -1;
    // the largest sizes do not overflow, and what lies beyond them is refused
    const int64_t big = (int64_t(1) << 31) - 1, wide = (int64_t(1) << 22) - 8;
    CHECK(gg_fp8_workspace_bytes(big, wide, 1) == size_t(big) * ((size_t(1) << 22) + (size_t(1) << 15)));
    CHECK(gg_fp8_glu_workspace_bytes(big, 256, 1 << 20, 1) > size_t(big) << 21);
    CHECK(gg_fp8_glu_workspace_bytes(1, 256, int64_t(1) << 62, 1) == 0 && gg_fp8_glu_workspace_bytes(1, 256, -8, 0) == 0);
    CHECK(gg_fp8_packed_bytes(GG_MAX_EXPERTS, 131072, 16256, 1) == size_t(1024) * (size_t(131072) * 16256 + 128 * 1024));   // 1024 row blocks of 127 scales in whole dwords
    CHECK(gg_fp8_packed_bytes(1, 131072, 16384, 1) == 0);
    CHECK(gg_fp8_glu_forward(x.p, off.as<int64_t>(), M, fc1.p, fc2.p, E, H, int64_t(1) << 62, 0, ws.p, need, nullptr, y.p, s) ==
          GG_ERR_INVALID_ARGUMENT);
}

// The tiles chosen at the sizes of tests/test_gpu_fp8_large.py and test_gpu_fp8.py, and the limits of streaming.
static void test_plan() {
    auto is = [](gg::F8Plan p, int rows, int columns, int group) {
        return p.rows == rows && p.columns == columns && p.group == group;
    };
    CHECK(is(gg::f8_plan(3445, 3, 16, 32, 3, 256), 256, 256, 64));       // few experts: 256 x 256
    CHECK(is(gg::f8_plan(3445, 3, 17, 33, 9, 256), 256, 256, 64));
    CHECK(is(gg::f8_plan(3438, 3, 16, 0, 9, 256), 256, 256, 64));        // gate and up (F 2040), dA (F 3968)
    CHECK(is(gg::f8_plan(3438, 3, 31, 0, 9, 256), 256, 256, 64));        // gate and up (F 3968)
    CHECK(is(gg::f8_plan(3438, 3, 8, 0, 9, 256), 128, 256, 64));         // dA (F 2040)
    CHECK(is(gg::f8_plan(4108, 12, 16, 32, 3, 256), 128, 256, 64));      // many: 128 x 256
    CHECK(is(gg::f8_plan(546, 9, 1, 2, 3, 256), 128, 128, 64));          // little work: 128 x 128
    CHECK(is(gg::f8_plan(64, 9, 1, 2, 3, 256), 0, 0, 64) && is(gg::f8_plan(65, 1, 1, 2, 3, 256), 128, 128, 64));
    CHECK(is(gg::f8_plan(1, 1, 16, 32, 16, 256), 0, 0, 64) && is(gg::f8_plan(1, 1, 16, 32, 17, 256), 0, 0, 32));
    CHECK(gg::f8_plan(1, 1, 16, 32, 32, 256).group == 32 && gg::f8_plan(1, 1, 16, 32, 33, 256).group == 0);
    CHECK(gg::f8_plan(1, 1, 16, 32, 33, 256).rows == 128);               // too wide to stream
    CHECK(gg::f8_plan(2147483647, 1024, 16384, 32767, 32767, 256).rows == 256);
}

static void test_debug_offsets_and_errors() {
    const int64_t E = 3, H = 64, F = 64, M = 8;
    Buf x(M * H * 2), off((E + 1) * 8), fc1(gg_fp8_packed_bytes(E, 2 * F, H, 2)), fc2(gg_fp8_packed_bytes(E, H, F, 1)), y(M * H * 2);
    Buf ws(gg_fp8_glu_workspace_bytes(M, H, F, 1)), h1(M * F * 4);
    const size_t need = gg_fp8_glu_workspace_bytes(M, H, F, 1);
    auto all = [&](hipStream_t st) {
        const int a = gg_fp8_forward(x.p, off.as<int64_t>(), M, fc2.p, E, H, F, 1, -1, nullptr, ws.p, need, y.p, st);
        const int b = gg_fp8_dgrad(x.p, nullptr, off.as<int64_t>(), M, fc2.p, E, H, F, 1, -1, nullptr, ws.p, need, y.p, st);
        const int c = gg_fp8_glu_forward(x.p, off.as<int64_t>(), M, fc1.p, fc2.p, E, H, F, 0, ws.p, need, nullptr, y.p, st);
        const int d = gg_fp8_glu_dgrad(x.p, h1.p, off.as<int64_t>(), M, fc1.p, fc2.p, E, H, F, 0, ws.p, need, y.p, st);
        CHECK(a == b && b == c && c == d);
        return a;
    };
    hipStream_t s = fake_stream(0);
    setenv("GG_DEBUG_VALIDATE", "1", 1);
    const int64_t good[] = {1, 1, 5, 8}, down[] = {0, 5, 4, 8}, over[] = {0, 1, 2, 9}, under[] = {-1, 0, 4, 8};
    const struct { const int64_t* o; int want; } sets[] = {{good, GG_OK}, {down, GG_ERR_INVALID_ARGUMENT},
                                                           {over, GG_ERR_INVALID_ARGUMENT},
                                                           {under, GG_ERR_INVALID_ARGUMENT}};
    for (const auto& t : sets) {
        for (int i = 0; i < 4; ++i) off.as<int64_t>()[i] = t.o[i];
        CHECK(all(s) == t.want);
    }
    unsetenv("GG_DEBUG_VALIDATE");
    CHECK(all(s) == GG_OK);   // not read on the host: the kernels keep wrong offsets in bounds
    fake_set_arch(2, "gfx942");
    CHECK(all(fake_stream(2)) == GG_ERR_UNSUPPORTED_DEVICE);
    fake_set_fail(1);
    CHECK(all(s) == GG_ERR_HIP);
    fake_set_fail(0);
    CHECK(all(s) == GG_OK);
}

int main() {
    test_products();
    test_block();
    test_plan();
    test_debug_offsets_and_errors();
    std::printf("%d of %d checks failed\n", g_failed, g_checked);
    return g_failed ? 1 : 0;
}
