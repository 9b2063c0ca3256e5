// C-ABI entry points of the block-scaled 8-bit floating-point expert products
// and the gated block made of them: argument validation and launches.
// Declarations and the contract are in include/gg.h.
//
// Every argument check runs before the first HIP call.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gg.h"
#include "gg_fp8.h"
#include "gg_host.h"

namespace {

using namespace gg;

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

int check_fp8_shape(int64_t M, int64_t E, int64_t N, int64_t K, int halves) {
    if (E < 1 || E > GG_MAX_EXPERTS || (halves != 1 && halves != 2)) return GG_ERR_INVALID_ARGUMENT;
    if (N <= 0 || K <= 0 || N % (8 * halves) != 0 || K % 8 != 0 || N >= (int64_t(1) << 22) || K >= (int64_t(1) << 22))
        return GG_ERR_INVALID_ARGUMENT;
    if (f8_matrix_bytes(f8_dim(N, halves), f8_dim(K, 1)) >= (int64_t(1) << 31)) return GG_ERR_INVALID_ARGUMENT;
    if (M < 0 || M >= (int64_t(1) << 31)) return GG_ERR_INVALID_ARGUMENT;
    return GG_OK;
}

// The gated block's sizes: W1 [2F][H], W2 [H][F].
int check_glu_shape(int64_t M, int64_t E, int64_t H, int64_t F) {
    if (F <= 0 || F >= (int64_t(1) << 22)) return GG_ERR_INVALID_ARGUMENT;     // 2F does not overflow
    return check_fp8_shape(M, E, 2 * F, H, 2);
}

size_t packed_bytes_of(int64_t E, const F8Dim& rows, const F8Dim& cont) {
    return static_cast<size_t>(E) * (f8_matrix_bytes(rows, cont) + f8_scale_bytes(rows, cont));
}

// The product of quantized rows by the packed matrices [rows][cont].
F8Params product(const uint8_t* q, const int64_t* offsets, int64_t M, const void* packed, int64_t E, const F8Dim& rows,
                 const F8Dim& cont, void* out) {
    F8Params g{};
    g.q = q;
    g.s = q + M * cont.padded();
    g.offsets = offsets;
    g.w = static_cast<const uint8_t*>(packed);
    g.w_stride = f8_matrix_bytes(rows, cont);
    g.ws = g.w + E * g.w_stride;
    g.ws_stride = f8_scale_bytes(rows, cont);
    g.ws_ld = f8_scale_ld(cont);
    g.M = static_cast<int>(M);
    g.E = static_cast<int>(E);
    g.kblocks = cont.blocks();
    g.n = rows;
    g.out = static_cast<uint16_t*>(out);
    return g;
}

F8QuantParams quantization(const void* x, const void* h1, const int64_t* offsets, int64_t M, int64_t E, const F8Dim& dim,
                           float slope, void* v_out, uint8_t* q) {
    F8QuantParams p{};
    p.x = static_cast<const uint16_t*>(x);
    p.h1 = static_cast<const uint16_t*>(h1);
    p.offsets = offsets;
    p.M = static_cast<int>(M);
    p.E = static_cast<int>(E);
    p.dim = dim;
    p.slope = slope;
    p.v_out = static_cast<uint16_t*>(v_out);
    p.q = q;
    p.s = q + M * dim.padded();
    return p;
}

int quantize_and_multiply(F8Mode mode, F8Epilogue epilogue, const F8QuantParams& p, F8Params g, int num_cu,
                          hipStream_t stream) {
    if (mode == F8_PLAIN && f8_quantizes(p.M, p.E, p.dim)) {
        g.x = p.x;
        g.k = p.dim;
    } else if (launch_f8_quant(mode, p, num_cu, stream) != hipSuccess) {
        return GG_ERR_HIP;
    }
    return launch_f8_gemm(epilogue, g, num_cu, stream) == hipSuccess ? GG_OK : GG_ERR_HIP;
}

// Whether a product's sums are fp32's: as asked for, else where its result is quantized again (it is not the last one).
bool sums_known(int sums) { return sums >= GG_FP8_SUMS_DEFAULT && sums <= GG_FP8_SUMS_SCALED; }
int fp32_sums(int sums, bool last) { return sums == GG_FP8_SUMS_FP32 || (sums == GG_FP8_SUMS_DEFAULT && !last); }

// Quantized rows start on 256 bytes.
size_t glu_rows(int64_t M, const F8Dim& d) { return (static_cast<size_t>(f8_rows_bytes(M, d)) + 255) / 256 * 256; }

}  // namespace

extern "C" {

size_t gg_fp8_scale_bytes(int64_t E, int64_t N, int64_t K, int halves) {
    if (check_fp8_shape(0, E, N, K, halves) != GG_OK) return 0;
    return static_cast<size_t>(E) * f8_dim(N, halves).blocks() * f8_dim(K, 1).blocks();
}

int gg_fp8_quantize_weights(const void* w, int64_t E, int64_t N, int64_t K, int halves, uint8_t* q, uint8_t* s,
                            hipStream_t stream) {
    int st = check_fp8_shape(0, E, N, K, halves);
    if (st != GG_OK) return st;
    if (!w || !q || !s) return GG_ERR_INVALID_ARGUMENT;
    if (!aligned16(w) || !aligned8(q)) return GG_ERR_MISALIGNED;
    st = check_aliasing({range_of(w, E * N * K * 2)}, {range_of(q, E * N * K), range_of(s, gg_fp8_scale_bytes(E, N, K, halves))});
    if (st != GG_OK) return st;
    DeviceInfo info;
    if ((st = device_info(stream, &info)) != GG_OK) return st;
    return launch_f8_quant_weights(static_cast<const uint16_t*>(w), static_cast<int>(E), f8_dim(N, halves), f8_dim(K, 1), q, s,
                                   stream) == hipSuccess
               ? GG_OK
               : GG_ERR_HIP;
}

size_t gg_fp8_packed_bytes(int64_t E, int64_t N, int64_t K, int halves) {
    if (check_fp8_shape(0, E, N, K, halves) != GG_OK) return 0;
    const size_t plain = packed_bytes_of(E, f8_dim(N, halves), f8_dim(K, 1));
    const size_t transposed = packed_bytes_of(E, f8_dim(K, 1), f8_dim(N, halves));
    return plain > transposed ? plain : transposed;   // they differ in the scales' padding
}

int gg_fp8_pack(const uint8_t* q, const uint8_t* s, int64_t E, int64_t N, int64_t K, int halves, int transposed,
                void* packed, size_t packed_bytes, hipStream_t stream) {
    int st = check_fp8_shape(0, E, N, K, halves);
    if (st != GG_OK) return st;
    if (!q || !s || !packed) return GG_ERR_INVALID_ARGUMENT;
    if (!aligned16(packed) || !aligned8(q)) return GG_ERR_MISALIGNED;
    const size_t need = gg_fp8_packed_bytes(E, N, K, halves);
    if (packed_bytes < need) return GG_ERR_WORKSPACE_TOO_SMALL;
    st = check_aliasing({range_of(q, E * N * K), range_of(s, gg_fp8_scale_bytes(E, N, K, halves))}, {range_of(packed, need)});
    if (st != GG_OK) return st;
    DeviceInfo info;
    if ((st = device_info(stream, &info)) != GG_OK) return st;
    return launch_f8_pack(q, s, static_cast<int>(E), f8_dim(N, halves), f8_dim(K, 1), transposed != 0,
                          static_cast<uint8_t*>(packed), stream) == hipSuccess
               ? GG_OK
               : GG_ERR_HIP;
}

size_t gg_fp8_workspace_bytes(int64_t M, int64_t width, int halves) {
    if (check_fp8_shape(M, 1, width, 8, halves) != GG_OK) return 0;
    return static_cast<size_t>(f8_rows_bytes(M, f8_dim(width, halves)));
}

int gg_fp8_forward(const void* x, const int64_t* offsets, int64_t M, const void* packed, int64_t E, int64_t N,
                   int64_t K, int halves, int activation, void* a_out, void* workspace, size_t workspace_bytes, void* y,
                   hipStream_t stream) {
    return gg_fp8_forward_sums(x, offsets, M, packed, E, N, K, halves, activation, a_out, workspace, workspace_bytes, y,
                               GG_FP8_SUMS_DEFAULT, stream);
}

int gg_fp8_forward_sums(const void* x, const int64_t* offsets, int64_t M, const void* packed, int64_t E, int64_t N,
                        int64_t K, int halves, int activation, void* a_out, void* workspace, size_t workspace_bytes,
                        void* y, int sums, hipStream_t stream) {
    int st = check_fp8_shape(M, E, N, K, halves);
    if (st != GG_OK) return st;
    if (!sums_known(sums)) return GG_ERR_INVALID_ARGUMENT;
    const bool glu = activation != GG_ACT_NONE;
    const float slope = glu ? act_slope(activation) : 1.0f;
    if (slope == 0.0f || (!glu && a_out)) return GG_ERR_INVALID_ARGUMENT;
    if (M == 0) return GG_OK;
    if (!x || !offsets || !packed || !workspace || !y) return GG_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(packed) || !aligned16(workspace) || !aligned16(y) || (a_out && !aligned16(a_out)) ||
        !aligned8(offsets))
        return GG_ERR_MISALIGNED;
    const size_t ws_need = gg_fp8_workspace_bytes(M, K, 1);
    if (workspace_bytes < ws_need) return GG_ERR_WORKSPACE_TOO_SMALL;
    st = check_aliasing({range_of(x, M * K * (glu ? 4 : 2)), range_of(offsets, (E + 1) * 8),
                         range_of(packed, gg_fp8_packed_bytes(E, N, K, halves))},
                        {range_of(y, M * N * 2), range_of(workspace, ws_need), range_of(a_out, a_out ? M * K * 2 : 0)});
    if (st != GG_OK) return st;
    DeviceInfo info;
    if ((st = device_info(stream, &info)) != GG_OK) return st;
    if ((st = debug_validate_offsets(offsets, E, M, stream)) != GG_OK) return st;
    uint8_t* q = static_cast<uint8_t*>(workspace);
    const F8Dim n = f8_dim(N, halves), k = f8_dim(K, 1);
    F8Params g = product(q, offsets, M, packed, E, n, k, y);
    g.fp32_sums = fp32_sums(sums, halves == 1);
    return quantize_and_multiply(glu ? F8_GLU : F8_PLAIN, F8_STORE, quantization(x, nullptr, offsets, M, E, k, slope, a_out, q),
                                 g, info.num_cu, stream);
}

int gg_fp8_dgrad(const void* dy, const void* h1, const int64_t* offsets, int64_t M, const void* packed, int64_t E,
                 int64_t N, int64_t K, int halves, int activation, void* dh1_out, void* workspace,
                 size_t workspace_bytes, void* dx, hipStream_t stream) {
    return gg_fp8_dgrad_sums(dy, h1, offsets, M, packed, E, N, K, halves, activation, dh1_out, workspace, workspace_bytes,
                             dx, GG_FP8_SUMS_DEFAULT, stream);
}

int gg_fp8_dgrad_sums(const void* dy, const void* h1, const int64_t* offsets, int64_t M, const void* packed, int64_t E,
                      int64_t N, int64_t K, int halves, int activation, void* dh1_out, void* workspace,
                      size_t workspace_bytes, void* dx, int sums, hipStream_t stream) {
    int st = check_fp8_shape(M, E, N, K, halves);
    if (st != GG_OK) return st;
    if (!sums_known(sums)) return GG_ERR_INVALID_ARGUMENT;
    const bool glu = activation != GG_ACT_NONE;
    const float slope = glu ? act_slope(activation) : 1.0f;
    if (slope == 0.0f || (glu && halves != 2) || (!glu && (h1 || dh1_out))) return GG_ERR_INVALID_ARGUMENT;
    if (M == 0) return GG_OK;
    if (!dy || (glu && !h1) || !offsets || !packed || !workspace || !dx) return GG_ERR_INVALID_ARGUMENT;
    if (!aligned16(dy) || (h1 && !aligned16(h1)) || !aligned16(packed) || !aligned16(workspace) || !aligned16(dx) ||
        (dh1_out && !aligned16(dh1_out)) || !aligned8(offsets))
        return GG_ERR_MISALIGNED;
    const size_t ws_need = gg_fp8_workspace_bytes(M, N, halves);
    if (workspace_bytes < ws_need) return GG_ERR_WORKSPACE_TOO_SMALL;
    st = check_aliasing({range_of(dy, M * N * (glu ? 1 : 2)), range_of(h1, h1 ? M * N * 2 : 0),
                         range_of(offsets, (E + 1) * 8), range_of(packed, gg_fp8_packed_bytes(E, N, K, halves))},
                        {range_of(dx, M * K * 2), range_of(workspace, ws_need),
                         range_of(dh1_out, dh1_out ? M * N * 2 : 0)});
    if (st != GG_OK) return st;
    DeviceInfo info;
    if ((st = device_info(stream, &info)) != GG_OK) return st;
    if ((st = debug_validate_offsets(offsets, E, M, stream)) != GG_OK) return st;
    uint8_t* q = static_cast<uint8_t*>(workspace);
    const F8Dim n = f8_dim(N, halves), k = f8_dim(K, 1);
    F8Params g = product(q, offsets, M, packed, E, k, n, dx);
    g.fp32_sums = fp32_sums(sums, halves == 2);
    return quantize_and_multiply(glu ? F8_DGLU : F8_PLAIN, F8_STORE, quantization(dy, h1, offsets, M, E, n, slope, dh1_out, q),
                                 g, info.num_cu, stream);
}

size_t gg_fp8_glu_workspace_bytes(int64_t M, int64_t H, int64_t F, int dgrad) {
    if (M == 0 || check_glu_shape(M, 1, H, F) != GG_OK) return 0;
    return glu_rows(M, f8_dim(H, 1)) + glu_rows(M, f8_dim(dgrad ? 2 * F : F, dgrad ? 2 : 1));
}

int gg_fp8_glu_forward(const void* x, const int64_t* offsets, int64_t M, const void* fc1, const void* fc2, int64_t E,
                       int64_t H, int64_t F, int activation, void* workspace, size_t workspace_bytes, void* h1_out,
                       void* y, hipStream_t stream) {
    return gg_fp8_glu_forward_sums(x, offsets, M, fc1, fc2, E, H, F, activation, workspace, workspace_bytes, h1_out, y,
                                   GG_FP8_SUMS_DEFAULT, stream);
}

int gg_fp8_glu_forward_sums(const void* x, const int64_t* offsets, int64_t M, const void* fc1, const void* fc2,
                            int64_t E, int64_t H, int64_t F, int activation, void* workspace, size_t workspace_bytes,
                            void* h1_out, void* y, int sums, hipStream_t stream) {
    int st = check_glu_shape(M, E, H, F);
    if (st != GG_OK) return st;
    if (!sums_known(sums)) return GG_ERR_INVALID_ARGUMENT;
    const float slope = act_slope(activation);
    if (slope == 0.0f) return GG_ERR_INVALID_ARGUMENT;
    if (M == 0) return GG_OK;
    if (!x || !offsets || !fc1 || !fc2 || !workspace || !y) return GG_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(fc1) || !aligned16(fc2) || !aligned16(workspace) || !aligned16(y) ||
        (h1_out && !aligned16(h1_out)) || !aligned8(offsets))
        return GG_ERR_MISALIGNED;
    const size_t ws_need = gg_fp8_glu_workspace_bytes(M, H, F, 0);
    if (workspace_bytes < ws_need) return GG_ERR_WORKSPACE_TOO_SMALL;
    st = check_aliasing({range_of(x, M * H * 2), range_of(offsets, (E + 1) * 8),
                         range_of(fc1, gg_fp8_packed_bytes(E, 2 * F, H, 2)), range_of(fc2, gg_fp8_packed_bytes(E, H, F, 1))},
                        {range_of(y, M * H * 2), range_of(workspace, ws_need), range_of(h1_out, h1_out ? M * F * 4 : 0)});
    if (st != GG_OK) return st;
    DeviceInfo info;
    if ((st = device_info(stream, &info)) != GG_OK) return st;
    if ((st = debug_validate_offsets(offsets, E, M, stream)) != GG_OK) return st;
    const F8Dim h = f8_dim(H, 1), f2 = f8_dim(2 * F, 2), f = f8_dim(F, 1);
    uint8_t *qx = static_cast<uint8_t*>(workspace), *qa = qx + glu_rows(M, h);
    F8Params g = product(qx, offsets, M, fc1, E, f2, h, h1_out);
    g.slope = slope;
    g.fp32_sums = fp32_sums(sums, false);
    g.q_out = qa;
    g.s_out = qa + M * f.padded();
    st = quantize_and_multiply(F8_PLAIN, F8_STORE_GLU, quantization(x, nullptr, offsets, M, E, h, 1.0f, nullptr, qx), g, info.num_cu,
                               stream);
    if (st != GG_OK) return st;
    g = product(qa, offsets, M, fc2, E, h, f, y);
    g.fp32_sums = fp32_sums(sums, true);
    return launch_f8_gemm(F8_STORE, g, info.num_cu, stream) == hipSuccess ? GG_OK : GG_ERR_HIP;
}

int gg_fp8_glu_dgrad(const void* dy, const void* h1, const int64_t* offsets, int64_t M, const void* fc1_t,
                     const void* fc2_t, int64_t E, int64_t H, int64_t F, int activation, void* workspace,
                     size_t workspace_bytes, void* dx, hipStream_t stream) {
    return gg_fp8_glu_dgrad_sums(dy, h1, offsets, M, fc1_t, fc2_t, E, H, F, activation, workspace, workspace_bytes, dx,
                                 GG_FP8_SUMS_DEFAULT, stream);
}

int gg_fp8_glu_dgrad_sums(const void* dy, const void* h1, const int64_t* offsets, int64_t M, const void* fc1_t,
                          const void* fc2_t, int64_t E, int64_t H, int64_t F, int activation, void* workspace,
                          size_t workspace_bytes, void* dx, int sums, hipStream_t stream) {
    int st = check_glu_shape(M, E, H, F);
    if (st != GG_OK) return st;
    if (!sums_known(sums)) return GG_ERR_INVALID_ARGUMENT;
    const float slope = act_slope(activation);
    if (slope == 0.0f) return GG_ERR_INVALID_ARGUMENT;
    if (M == 0) return GG_OK;
    if (!dy || !h1 || !offsets || !fc1_t || !fc2_t || !workspace || !dx) return GG_ERR_INVALID_ARGUMENT;
    if (!aligned16(dy) || !aligned16(h1) || !aligned16(fc1_t) || !aligned16(fc2_t) || !aligned16(workspace) ||
        !aligned16(dx) || !aligned8(offsets))
        return GG_ERR_MISALIGNED;
    const size_t ws_need = gg_fp8_glu_workspace_bytes(M, H, F, 1);
    if (workspace_bytes < ws_need) return GG_ERR_WORKSPACE_TOO_SMALL;
    st = check_aliasing({range_of(dy, M * H * 2), range_of(h1, M * F * 4), range_of(offsets, (E + 1) * 8),
                         range_of(fc1_t, gg_fp8_packed_bytes(E, 2 * F, H, 2)),
                         range_of(fc2_t, gg_fp8_packed_bytes(E, H, F, 1))},
                        {range_of(dx, M * H * 2), range_of(workspace, ws_need)});
    if (st != GG_OK) return st;
    DeviceInfo info;
    if ((st = device_info(stream, &info)) != GG_OK) return st;
    if ((st = debug_validate_offsets(offsets, E, M, stream)) != GG_OK) return st;
    const F8Dim h = f8_dim(H, 1), f2 = f8_dim(2 * F, 2), f = f8_dim(F, 1);
    uint8_t *qy = static_cast<uint8_t*>(workspace), *qd = qy + glu_rows(M, h);
    F8Params g = product(qy, offsets, M, fc2_t, E, f, h, nullptr);
    g.h1 = static_cast<const uint16_t*>(h1);
    g.slope = slope;
    g.fp32_sums = fp32_sums(sums, false);
    g.q_out = qd;
    g.s_out = qd + M * f2.padded();
    st = quantize_and_multiply(F8_PLAIN, F8_STORE_DGLU, quantization(dy, nullptr, offsets, M, E, h, 1.0f, nullptr, qy), g, info.num_cu,
                               stream);
    if (st != GG_OK) return st;
    g = product(qd, offsets, M, fc1_t, E, h, f2, dx);
    g.fp32_sums = fp32_sums(sums, true);
    return launch_f8_gemm(F8_STORE, g, info.num_cu, stream) == hipSuccess ? GG_OK : GG_ERR_HIP;
}

}  // extern "C"
