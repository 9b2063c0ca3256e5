// C-ABI entry points of the 8-bit expert products: argument validation and
// launches.  Declarations and the contract are in include/gg.h.
//
// Every argument check runs before the first HIP call.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gg.h"
#include "gg_host.h"
#include "gg_int8.h"

namespace {

using namespace gg;

int check_int8_shape(int64_t M, int64_t E, int64_t N, int64_t K) {
    if (E < 1 || E > GG_MAX_EXPERTS) return GG_ERR_INVALID_ARGUMENT;
    if (N <= 0 || K <= 0 || N % 8 != 0 || K % 8 != 0 || N > GG_INT8_MAX_SUM || K > GG_INT8_MAX_SUM)
        return GG_ERR_INVALID_ARGUMENT;
    // the declared limit of one packed matrix; the kernels themselves address it with 64 bits
    if (i8_rows_p(N) * i8_cont_p(K) >= (int64_t(1) << 31) || i8_rows_p(K) * i8_cont_p(N) >= (int64_t(1) << 31))
        return GG_ERR_INVALID_ARGUMENT;
    if (M < 0 || M >= (int64_t(1) << 31)) return GG_ERR_INVALID_ARGUMENT;
    return GG_OK;
}

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

size_t matrix_bytes(int64_t rows, int64_t cont) { return static_cast<size_t>(i8_rows_p(rows)) * i8_cont_p(cont); }

// Quantize `p` into the workspace, then multiply by the packed matrix [out_cols][p.K].
int quantize_and_multiply(QuantMode mode, QuantParams p, const void* packed, int64_t out_cols, const float* ws, int ws_ld,
                          void* workspace, void* out, hipStream_t stream, int num_cu) {
    p.width = static_cast<int>(i8_cont_p(p.K));
    p.q = static_cast<int8_t*>(workspace);
    p.q_block = static_cast<int64_t>(p.M) * 64;
    p.q_row = 64;
    p.blocked = 1;
    p.s = reinterpret_cast<float*>(p.q + static_cast<int64_t>(p.M) * p.width);
    if (launch_quant_rows(mode, p, num_cu, stream) != hipSuccess) return GG_ERR_HIP;
    Int8Params g{};
    g.q = p.q;
    g.s = p.s;
    g.offsets = p.offsets;
    g.w = static_cast<const int8_t*>(packed);
    g.w_stride = static_cast<int64_t>(matrix_bytes(out_cols, p.K));
    g.ws = ws;
    g.ws_ld = ws_ld;
    g.width = p.width;
    g.M = p.M;
    g.E = p.E;
    g.N = static_cast<int>(out_cols);
    g.out = static_cast<uint16_t*>(out);
    return launch_int8_gemm(g, num_cu, stream) == hipSuccess ? GG_OK : GG_ERR_HIP;
}

}  // namespace

extern "C" {

int gg_int8_quantize_rows(const void* x, int64_t M, int64_t K, int8_t* q, float* s, hipStream_t stream) {
    if (M < 0 || M >= (int64_t(1) << 31) || K <= 0 || K % 8 != 0 || K >= (int64_t(1) << 22)) return GG_ERR_INVALID_ARGUMENT;
    if (M == 0) return GG_OK;
    if (!x || !q || !s) return GG_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned8(q) || !aligned4(s)) return GG_ERR_MISALIGNED;
    int st = check_aliasing({range_of(x, M * K * 2)}, {range_of(q, M * K), range_of(s, M * 4)});
    if (st != GG_OK) return st;
    DeviceInfo info;
    if ((st = device_info(stream, &info)) != GG_OK) return st;
    QuantParams p{};
    p.x = static_cast<const uint16_t*>(x);
    p.M = static_cast<int>(M);
    p.K = p.width = static_cast<int>(K);
    p.q = q;
    p.q_block = 64;
    p.q_row = K;
    p.s = s;
    return launch_quant_rows(Q_PLAIN, p, info.num_cu, stream) == hipSuccess ? GG_OK : GG_ERR_HIP;
}

size_t gg_int8_packed_bytes(int64_t E, int64_t N, int64_t K, int transposed) {
    if (check_int8_shape(0, E, N, K) != GG_OK) return 0;
    const size_t m = transposed ? matrix_bytes(K, N) : matrix_bytes(N, K);
    return static_cast<size_t>(E) * (m + 4 * static_cast<size_t>(i8_cont_p(N)));
}

int gg_int8_pack(const int8_t* wq, const float* ws, int64_t E, int64_t N, int64_t K, int transposed, void* packed,
                 size_t packed_bytes, hipStream_t stream) {
    int st = check_int8_shape(0, E, N, K);
    if (st != GG_OK) return st;
    if (!wq || !ws || !packed) return GG_ERR_INVALID_ARGUMENT;
    if (!aligned16(packed) || !aligned4(ws)) return GG_ERR_MISALIGNED;
    const size_t need = gg_int8_packed_bytes(E, N, K, transposed);
    if (packed_bytes < need) return GG_ERR_WORKSPACE_TOO_SMALL;
    if ((st = check_aliasing({range_of(wq, E * N * K), range_of(ws, E * N * 4)}, {range_of(packed, need)})) != GG_OK)
        return st;
    DeviceInfo info;
    if ((st = device_info(stream, &info)) != GG_OK) return st;
    return launch_int8_pack(wq, ws, static_cast<int>(E), static_cast<int>(N), static_cast<int>(K), transposed != 0,
                            static_cast<int8_t*>(packed), stream) == hipSuccess
               ? GG_OK
               : GG_ERR_HIP;
}

size_t gg_int8_workspace_bytes(int64_t M, int64_t width) {
    if (M <= 0 || width <= 0 || width > GG_INT8_MAX_SUM) return 0;
    return static_cast<size_t>(M) * (static_cast<size_t>(i8_cont_p(width)) + 4);
}

int gg_int8_forward(const void* x, const int64_t* offsets, int64_t M, const void* packed, int64_t E, int64_t N,
                    int64_t K, int activation, void* a_out, void* workspace, size_t workspace_bytes, void* y,
                    hipStream_t stream) {
    int st = check_int8_shape(M, E, N, K);
    if (st != GG_OK) return st;
    const bool glu = activation != GG_ACT_NONE;
    const float slope = glu ? act_slope(activation) : 1.0f;
    if (slope == 0.0f || (!glu && a_out)) return GG_ERR_INVALID_ARGUMENT;
    if (M == 0) return GG_OK;
    if (!x || !offsets || !packed || !workspace || !y) return GG_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(packed) || !aligned16(workspace) || !aligned16(y) || (a_out && !aligned16(a_out)) ||
        !aligned8(offsets))
        return GG_ERR_MISALIGNED;
    const size_t ws_need = gg_int8_workspace_bytes(M, K);
    if (workspace_bytes < ws_need) return GG_ERR_WORKSPACE_TOO_SMALL;
    st = check_aliasing({range_of(x, M * K * (glu ? 4 : 2)), range_of(offsets, (E + 1) * 8),
                         range_of(packed, gg_int8_packed_bytes(E, N, K, 0))},
                        {range_of(y, M * N * 2), range_of(workspace, ws_need), range_of(a_out, a_out ? M * K * 2 : 0)});
    if (st != GG_OK) return st;
    DeviceInfo info;
    if ((st = device_info(stream, &info)) != GG_OK) return st;
    if ((st = debug_validate_offsets(offsets, E, M, stream)) != GG_OK) return st;
    QuantParams p{};
    p.x = static_cast<const uint16_t*>(x);
    p.offsets = offsets;
    p.M = static_cast<int>(M);
    p.E = static_cast<int>(E);
    p.K = static_cast<int>(K);
    p.slope = slope;
    p.v_out = static_cast<uint16_t*>(a_out);
    const float* scales = reinterpret_cast<const float*>(static_cast<const char*>(packed) + E * matrix_bytes(N, K));
    return quantize_and_multiply(glu ? Q_GLU : Q_PLAIN, p, packed, N, scales, static_cast<int>(i8_cont_p(N)), workspace, y,
                                 stream, info.num_cu);
}

int gg_int8_dgrad(const void* dy, const void* h1, const int64_t* offsets, int64_t M, const void* packed, int64_t E,
                  int64_t N, int64_t K, int activation, void* dh1_out, void* workspace, size_t workspace_bytes,
                  void* dx, hipStream_t stream) {
    int st = check_int8_shape(M, E, N, K);
    if (st != GG_OK) return st;
    const bool glu = activation != GG_ACT_NONE;
    const float slope = glu ? act_slope(activation) : 1.0f;
    if (slope == 0.0f || (glu && N % 16 != 0) || (!glu && (h1 || dh1_out))) return GG_ERR_INVALID_ARGUMENT;
    if (M == 0) return GG_OK;
    if (!dy || (glu && !h1) || !offsets || !packed || !workspace || !dx) return GG_ERR_INVALID_ARGUMENT;
    if (!aligned16(dy) || (h1 && !aligned16(h1)) || !aligned16(packed) || !aligned16(workspace) || !aligned16(dx) ||
        (dh1_out && !aligned16(dh1_out)) || !aligned8(offsets))
        return GG_ERR_MISALIGNED;
    const size_t ws_need = gg_int8_workspace_bytes(M, N);
    if (workspace_bytes < ws_need) return GG_ERR_WORKSPACE_TOO_SMALL;
    st = check_aliasing({range_of(dy, M * N * (glu ? 1 : 2)), range_of(h1, h1 ? M * N * 2 : 0),
                         range_of(offsets, (E + 1) * 8), range_of(packed, gg_int8_packed_bytes(E, N, K, 1))},
                        {range_of(dx, M * K * 2), range_of(workspace, ws_need),
                         range_of(dh1_out, dh1_out ? M * N * 2 : 0)});
    if (st != GG_OK) return st;
    DeviceInfo info;
    if ((st = device_info(stream, &info)) != GG_OK) return st;
    if ((st = debug_validate_offsets(offsets, E, M, stream)) != GG_OK) return st;
    QuantParams p{};
    p.x = static_cast<const uint16_t*>(dy);
    p.h1 = static_cast<const uint16_t*>(h1);
    p.offsets = offsets;
    p.cs = reinterpret_cast<const float*>(static_cast<const char*>(packed) + E * matrix_bytes(K, N));
    p.cs_ld = static_cast<int>(i8_cont_p(N));
    p.M = static_cast<int>(M);
    p.E = static_cast<int>(E);
    p.K = static_cast<int>(N);
    p.slope = slope;
    p.v_out = static_cast<uint16_t*>(dh1_out);
    return quantize_and_multiply(glu ? Q_DGLU : Q_SCALED, p, packed, K, nullptr, 0, workspace, dx, stream, info.num_cu);
}

}  // extern "C"
