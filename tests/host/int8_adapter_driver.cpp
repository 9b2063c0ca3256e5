// Host-side driver of the C-ABI layer of the 8-bit products and the adapters
// (gg_int8_api.cpp, gg_adapter_api.cpp) built with the fake HIP runtime and
// the recording launchers below: the launches each entry point makes and
// their parameters, the workspace's layout, sizes at the largest allowed
// counts, device checks, runtime errors and the debug offset check.  Built and
// run under AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_host_sanitized_int8.py.  Exit status 0 when every check holds.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "fake_hip.h"
#include "gg.h"
#include "gg_adapter.h"
#include "gg_int8.h"

namespace {

struct Record {
    int kind;   // 0 quantize, 1 multiply, 2 pack, 3 adapter forward, 4 adapter backward
    gg::QuantMode mode;
    gg::QuantParams q;
    gg::Int8Params g;
    gg::AdapterParams a;
    int num_cu;
    hipStream_t stream;
};
std::vector<Record> g_rec;
hipError_t g_result = hipSuccess;
int g_fail_kind = -1;

hipError_t result(int kind) { return kind == g_fail_kind ? hipErrorLaunchFailure : g_result; }

}  // namespace

namespace gg {
hipError_t launch_quant_rows(QuantMode mode, const QuantParams& p, int num_cu, hipStream_t s) {
    Record r{};
    r.kind = 0, r.mode = mode, r.q = p, r.num_cu = num_cu, r.stream = s;
    g_rec.push_back(r);
    return result(0);
}
hipError_t launch_int8_gemm(const Int8Params& p, int num_cu, hipStream_t s) {
    Record r{};
    r.kind = 1, r.g = p, r.num_cu = num_cu, r.stream = s;
    g_rec.push_back(r);
    return result(1);
}
hipError_t launch_int8_pack(const int8_t*, const float*, int, int, int, int, int8_t*, hipStream_t s) {
    Record r{};
    r.kind = 2, r.stream = s;
    g_rec.push_back(r);
    return result(2);
}
hipError_t launch_adapter_forward(const AdapterParams& p, int num_cu, hipStream_t s) {
    Record r{};
    r.kind = 3, r.a = p, r.num_cu = num_cu, r.stream = s;
    g_rec.push_back(r);
    return result(3);
}
hipError_t launch_adapter_backward(const AdapterParams& p, int num_cu, hipStream_t s) {
    Record r{};
    r.kind = 4, r.a = p, r.num_cu = num_cu, r.stream = s;
    g_rec.push_back(r);
    return result(4);
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

static void test_int8() {
    const int64_t E = 3, N = 48, K = 264, M = 21;
    Buf x(M * 2 * K * 2), off((E + 1) * 8), w(gg_int8_packed_bytes(E, N, K, 0)), wt(gg_int8_packed_bytes(E, N, K, 1));
    Buf a(M * K * 2), y(M * N * 2), ws(gg_int8_workspace_bytes(M, K));
    off.as<int64_t>()[E] = M;
    hipStream_t s = fake_stream(0);
    g_rec.clear();
    CHECK(gg_int8_forward(x.p, off.as<int64_t>(), M, w.p, E, N, K, GG_ACT_QGEGLU, a.p, ws.p,
                          gg_int8_workspace_bytes(M, K), y.p, s) == GG_OK);
    CHECK(g_rec.size() == 2 && g_rec[0].kind == 0 && g_rec[1].kind == 1);
    const gg::QuantParams q = g_rec[0].q;
    CHECK(g_rec[0].mode == gg::Q_GLU && q.K == K && q.width == 384 && q.M == M && q.slope == 1.702f && q.blocked);
    CHECK(q.q == ws.as<int8_t>() && reinterpret_cast<int8_t*>(q.s) == q.q + M * 384 && q.v_out == a.as<uint16_t>());
    CHECK(reinterpret_cast<uint8_t*>(q.s + M) == ws.p + gg_int8_workspace_bytes(M, K));
    CHECK(q.q_block == M * 64 && q.q_row == 64);
    const gg::Int8Params g = g_rec[1].g;
    CHECK(g.q == q.q && g.s == q.s && g.N == N && g.width == 384 && g.w_stride == 64 * 384 && g.ws_ld == 128);
    CHECK(reinterpret_cast<const uint8_t*>(g.ws) == w.p + E * g.w_stride);
    CHECK(reinterpret_cast<const uint8_t*>(g.ws + E * g.ws_ld) == w.p + gg_int8_packed_bytes(E, N, K, 0));
    CHECK(g_rec[0].stream == s && g_rec[1].stream == s && g_rec[1].num_cu == 256);
    // the gradient: column scales go into the quantization, none into the product
    Buf h1(M * N * 2), dh(M * N * 2), dx(M * K * 2), ws2(gg_int8_workspace_bytes(M, N));
    g_rec.clear();
    CHECK(gg_int8_dgrad(y.p, h1.p, off.as<int64_t>(), M, wt.p, E, N, K, GG_ACT_SWIGLU, dh.p, ws2.p,
                        gg_int8_workspace_bytes(M, N), dx.p, s) == GG_OK);
    CHECK(g_rec.size() == 2 && g_rec[0].mode == gg::Q_DGLU && g_rec[0].q.h1 == h1.as<uint16_t>());
    CHECK(g_rec[0].q.K == N && g_rec[0].q.width == 128 && g_rec[0].q.cs_ld == 128);
    CHECK(reinterpret_cast<const uint8_t*>(g_rec[0].q.cs + E * 128) == wt.p + gg_int8_packed_bytes(E, N, K, 1));
    CHECK(g_rec[1].g.ws == nullptr && g_rec[1].g.N == K && g_rec[1].g.w_stride == 288 * 128);
    g_rec.clear();
    CHECK(gg_int8_dgrad(y.p, nullptr, off.as<int64_t>(), M, wt.p, E, N, K, GG_ACT_NONE, nullptr, ws2.p,
                        gg_int8_workspace_bytes(M, N), dx.p, s) == GG_OK);
    CHECK(g_rec.size() == 2 && g_rec[0].mode == gg::Q_SCALED && !g_rec[0].q.h1 && !g_rec[0].q.v_out);
    // quantization alone keeps the caller's layout
    Buf qo(M * K), so(M * 4);
    g_rec.clear();
    CHECK(gg_int8_quantize_rows(x.p, M, K, qo.as<int8_t>(), so.as<float>(), s) == GG_OK);
    CHECK(g_rec.size() == 1 && g_rec[0].mode == gg::Q_PLAIN && g_rec[0].q.width == K && !g_rec[0].q.blocked);
    CHECK(g_rec[0].q.q_row == K && !g_rec[0].q.offsets);
    // no rows: success, no launch
    g_rec.clear();
    CHECK(gg_int8_forward(nullptr, nullptr, 0, nullptr, E, N, K, -1, nullptr, nullptr, 0, nullptr, s) == GG_OK);
    CHECK(g_rec.empty());
    // a launch that fails is an error, and nothing follows it
    g_fail_kind = 0;
    CHECK(gg_int8_forward(x.p, off.as<int64_t>(), M, w.p, E, N, K, -1, nullptr, ws.p, gg_int8_workspace_bytes(M, K), y.p,
                          s) == GG_ERR_HIP);
    CHECK(g_rec.size() == 1);
    g_fail_kind = 1;
    CHECK(gg_int8_forward(x.p, off.as<int64_t>(), M, w.p, E, N, K, -1, nullptr, ws.p, gg_int8_workspace_bytes(M, K), y.p,
                          s) == GG_ERR_HIP);
    g_fail_kind = 2;
    Buf wq(E * N * K), wsc(E * N * 4);
    CHECK(gg_int8_pack(wq.as<int8_t>(), wsc.as<float>(), E, N, K, 1, wt.p, gg_int8_packed_bytes(E, N, K, 1), s) ==
          GG_ERR_HIP);
    g_fail_kind = -1;
    // the largest sizes do not overflow
    CHECK(gg_int8_workspace_bytes((int64_t(1) << 31) - 1, GG_INT8_MAX_SUM) == ((size_t(1) << 31) - 1) * (131072 + 4));
    CHECK(gg_int8_packed_bytes(GG_MAX_EXPERTS, 131072, 16256, 0) == size_t(1024) * (size_t(131072) * 16256 + 4 * 131072));
    CHECK(gg_int8_packed_bytes(1, 131072, 16384, 0) == 0 && gg_int8_packed_bytes(1, 16384, 131072, 0) == 0);
}

static void test_adapter() {
    const int64_t E = 3, N = 2056, K = 520, r = 40, M = 1500;
    const size_t need = gg_adapter_workspace_bytes(M, E, N, K, r);
    Buf x(M * K * 2), dy(M * N * 2), u(M * r * 2), off((E + 1) * 8), a(E * r * K * 2), b(E * N * r * 2), y(M * N * 2);
    Buf dx(M * K * 2), da(E * r * K * 4), db(E * N * r * 4), ws(need);
    off.as<int64_t>()[E] = M;
    hipStream_t s = fake_stream(0);
    g_rec.clear();
    // the base may be the output itself
    CHECK(gg_adapter_forward(x.p, off.as<int64_t>(), M, a.p, b.p, E, N, K, r, 0.5f, y.p, u.p, y.p, s) == GG_OK);
    CHECK(g_rec.size() == 1 && g_rec[0].kind == 3 && g_rec[0].a.base == g_rec[0].a.out && g_rec[0].a.scale == 0.5f);
    CHECK(gg_adapter_forward(x.p, off.as<int64_t>(), M, a.p, b.p, E, N, K, r, 0.5f, x.p, u.p, y.p, s) == GG_OK);
    g_rec.clear();
    CHECK(gg_adapter_backward(dy.p, x.p, u.p, off.as<int64_t>(), M, a.p, b.p, E, N, K, r, 0.5f, nullptr, ws.p, need, dx.p,
                              da.as<float>(), db.as<float>(), 7, s) == GG_OK);
    CHECK(g_rec.size() == 1 && g_rec[0].kind == 4);
    const gg::AdapterParams p = g_rec[0].a;
    const int64_t rp = 64, chunks = 5, blocks = 1500 / 32 + 3;   // 4 x 128 columns a chunk at rank 33 .. 64
    CHECK(p.accumulate == 1 && p.blocks == blocks && p.rows1 % 32 == 0 && p.rows2 % 32 == 0);
    CHECK(p.rows1 >= 256 && p.rows2 >= 256);
    auto at = [&](const void* q) { return reinterpret_cast<const uint8_t*>(q) - ws.p; };
    CHECK(at(p.du_part) == 0 && at(p.du) >= chunks * blocks * 32 * rp * 4);
    CHECK(at(p.du_t) - at(p.du) >= blocks * 32 * rp * 2 && at(p.db_part) - at(p.du_t) >= blocks * 32 * rp * 6);
    CHECK(at(p.da_part) - at(p.db_part) >= (2 * M / p.rows1) * N * r * 4);
    CHECK(int64_t(need) - at(p.da_part) >= (2 * M / p.rows2) * K * r * 4);
    for (const void* q : {(const void*)p.du_part, (const void*)p.du, (const void*)p.du_t, (const void*)p.db_part,
                          (const void*)p.da_part})
        CHECK(at(q) % 256 == 0);
    // no rows: the gradients are still written (or kept, to add to)
    g_rec.clear();
    CHECK(gg_adapter_backward(nullptr, nullptr, nullptr, off.as<int64_t>(), 0, nullptr, nullptr, E, N, K, r, 1.0f, nullptr,
                              nullptr, 0, nullptr, da.as<float>(), db.as<float>(), 0, s) == GG_OK);
    CHECK(g_rec.size() == 1 && g_rec[0].a.M == 0 && g_rec[0].a.blocks == 0);
    g_fail_kind = 4;
    CHECK(gg_adapter_backward(dy.p, x.p, u.p, off.as<int64_t>(), M, a.p, b.p, E, N, K, r, 0.5f, nullptr, ws.p, need, dx.p,
                              da.as<float>(), db.as<float>(), 0, s) == GG_ERR_HIP);
    g_fail_kind = -1;
    // the largest counts: sizes stay positive and a unit's rows stay within 32 bits
    const int64_t big = (int64_t(1) << 31) - 1;
    const size_t huge = gg_adapter_workspace_bytes(big, GG_MAX_EXPERTS, (int64_t(1) << 22) - 8, 8, 64);
    CHECK(huge > size_t(big) * 64 * 4 * 8191 && huge < (size_t(1) << 62));
    g_rec.clear();
    uint8_t* const far = reinterpret_cast<uint8_t*>(uintptr_t(1) << 40);   // addresses only: nothing reads them here
    const int64_t n2 = (int64_t(1) << 22) - 8;
    CHECK(gg_adapter_backward(far, far + (size_t(1) << 56), far + (size_t(2) << 56), off.as<int64_t>(), big, a.p, b.p, 1,
                              n2, 8, 64, 1.0f, nullptr, far + (size_t(3) << 56), huge, far + (size_t(8) << 56),
                              reinterpret_cast<float*>(far + (size_t(9) << 56)),
                              reinterpret_cast<float*>(far + (size_t(10) << 56)), 0, s) == GG_OK);
    CHECK(g_rec.size() == 1 && g_rec[0].a.rows1 > 0 && g_rec[0].a.rows1 % 32 == 0 && g_rec[0].a.rows2 > 0);
}

static void test_debug_offsets_and_errors() {
    const int64_t E = 3, N = 64, K = 64, M = 8;
    Buf x(M * K * 2), off((E + 1) * 8), w(gg_int8_packed_bytes(E, N, K, 0)), y(M * N * 2);
    Buf ws(gg_int8_workspace_bytes(M, K)), a(E * 8 * K * 2), b(E * N * 8 * 2), u(M * 8 * 2);
    hipStream_t s = fake_stream(0);
    auto both = [&](hipStream_t st) {
        const int q = gg_int8_forward(x.p, off.as<int64_t>(), M, w.p, E, N, K, -1, nullptr, ws.p,
                                      gg_int8_workspace_bytes(M, K), y.p, st);
        const int f = gg_adapter_forward(x.p, off.as<int64_t>(), M, a.p, b.p, E, N, K, 8, 1.0f, nullptr, u.p, y.p, st);
        CHECK(q == f);
        return q;
    };
    setenv("GG_DEBUG_VALIDATE", "1", 1);
    const int64_t good[] = {1, 1, 5, 8}, down[] = {0, 5, 4, 8}, over[] = {0, 1, 2, 9}, under[] = {-1, 0, 4, 8};
    const struct { const int64_t* o; int want; } sets[] = {{good, GG_OK}, {down, GG_ERR_INVALID_ARGUMENT},
                                                           {over, GG_ERR_INVALID_ARGUMENT},
                                                           {under, GG_ERR_INVALID_ARGUMENT}};
    for (const auto& t : sets) {
        for (int i = 0; i < 4; ++i) off.as<int64_t>()[i] = t.o[i];
        CHECK(both(s) == t.want);
    }
    unsetenv("GG_DEBUG_VALIDATE");
    CHECK(both(s) == GG_OK);   // not read on the host: the kernels keep wrong offsets in bounds
    // a device of another architecture, and a runtime that fails
    fake_set_arch(2, "gfx942");
    CHECK(both(fake_stream(2)) == GG_ERR_UNSUPPORTED_DEVICE);
    fake_set_fail(1);
    CHECK(both(s) == GG_ERR_HIP);
    fake_set_fail(0);
    CHECK(both(s) == GG_OK);
}

int main() {
    test_int8();
    test_adapter();
    test_debug_offsets_and_errors();
    std::printf("%d of %d checks failed\n", g_failed, g_checked);
    return g_failed ? 1 : 0;
}
