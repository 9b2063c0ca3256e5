// Internal interface between the C-ABI entry points of the block-scaled 8-bit
// floating-point products (gg_fp8_api.cpp) and their kernels (gg_fp8.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

namespace gg {

constexpr int F8_BLOCK = 128;   // values that share a scale

// One dimension of a matrix: one part, or two equal halves (gate, up), each
// padded to whole blocks, so that no block holds values of both.
struct F8Dim {
    int part, part_p, parts;   // real and padded values of a part
    __host__ __device__ int real() const { return part * parts; }
    __host__ __device__ int padded() const { return part_p * parts; }
    __host__ __device__ int blocks() const { return padded() / F8_BLOCK; }
};
inline F8Dim f8_dim(int64_t n, int parts) {
    const int64_t part = n / parts;
    return F8Dim{static_cast<int>(part), static_cast<int>((part + F8_BLOCK - 1) / F8_BLOCK * F8_BLOCK), parts};
}

// Layouts.  Quantized rows: 64-byte blocks, column c (padded) of row r at
// (c / 64) * 64 M + 64 r + c % 64; their scales, a byte each (2^(byte - 127)),
// four blocks of a row in a dword: block k of row r at 4 ((k / 4) M + r) + k % 4.
// A packed matrix [rows][cont] (rows: output columns of the product, cont: the
// summed dimension): 32-row blocks, each of cont_p / 64 steps of 2 KiB in the
// operand order of the 32x32x64 matrix instruction: lane l holds row
// 32 b + (l & 31), columns 64 s + 32 (l >> 5) onwards, 32 of them, as two
// 16-byte operands 1 KiB apart.  Its scales: for each 128 rows, a byte for each
// block of cont, in whole dwords.
inline int64_t f8_matrix_bytes(const F8Dim& rows, const F8Dim& cont) {
    return static_cast<int64_t>(rows.padded()) * cont.padded();
}
__host__ __device__ inline int f8_scale_ld(const F8Dim& cont) { return (cont.blocks() + 3) / 4 * 4; }
inline int64_t f8_scale_bytes(const F8Dim& rows, const F8Dim& cont) {
    return static_cast<int64_t>(rows.blocks()) * f8_scale_ld(cont);
}
inline int64_t f8_rows_bytes(int64_t M, const F8Dim& cont) {
    return M * (cont.padded() + f8_scale_ld(cont));
}

// What a row's 8-bit values are made from.
enum F8Mode {
    F8_PLAIN = 0,   // v = x
    F8_GLU = 1,     // v = bf16(act(gate) * up) of x = [gate | up]
    F8_DGLU = 2     // v = bf16(derivative of the activation at h1, times x)
};

struct F8QuantParams {
    const uint16_t* x;       // [M][dim] bf16 (F8_GLU: [M][2 dim], F8_DGLU: [M][dim / 2])
    const uint16_t* h1;      // F8_DGLU: [M][dim]
    const int64_t* offsets;  // [E+1]
    int M, E;
    F8Dim dim;               // a quantized row (F8_DGLU: two parts)
    float slope;
    uint16_t* v_out;         // F8_GLU, F8_DGLU: v [M][dim], or null
    uint8_t* q;
    uint8_t* s;
};

// What becomes of a product's sums acc[r][n] = sum_k v[r][k] W_e[n][k].
enum F8Epilogue {
    F8_STORE = 0,       // out = bf16(acc)
    F8_STORE_GLU = 1,   // n: two parts, H1 = bf16(acc) (stored where h1_out is given); A = bf16(act(gate) * up), quantized
    F8_STORE_DGLU = 2   // dA = bf16(acc), dH1 = bf16(derivative at h1, times dA), quantized
};

struct F8Params {
    const uint8_t* q;        // quantized rows
    const uint8_t* s;        // and their scales
    const int64_t* offsets;  // [E+1]
    const uint8_t* w;        // packed matrices
    int64_t w_stride;        // bytes of one expert's matrix
    const uint8_t* ws;       // and their scales
    int64_t ws_stride;       // bytes of one expert's scales
    int ws_ld;               // bytes of the scales of 128 rows
    int M, E;
    int kblocks;             // blocks of the summed dimension
    F8Dim n;                 // columns
    const uint16_t* x;       // rows [M][k] to be quantized by the product itself (f8_quantizes), or null
    F8Dim k;                 // with x: the summed dimension
    uint16_t* out;           // F8_STORE: [M][n]; F8_STORE_GLU: H1 [M][n], or null
    const uint16_t* h1;      // F8_STORE_DGLU: [M][2 n]
    float slope;
    uint8_t* q_out;          // A or dH1, quantized
    uint8_t* s_out;
    int tile;                // whether there are tiles (set by the launcher)
    int group;               // rows of a streaming item, at most; 0: there are none (set by the launcher)
    int fp32_sums;           // sums in fp32 (operands as bf16), or the scaled 8-bit instruction's
};

constexpr int F8_GROUP = 64;                    // rows of a streaming item, at most
constexpr int F8_PANEL = 128 * 1024;            // LDS for a streaming item's rows
constexpr int F8_RING = F8_PANEL + 4 * 1024;    // LDS for operands

// Which tiles a product of M rows over E experts takes (0 rows: none), and how many rows a streaming item has at most
// (0: there are none; what 128 KiB hold of the summed width).  wide, narrow: tiles of 256 and of 128 packed columns
// side by side (narrow 0: there is no such kernel).
//
// Up to 64 rows in all are streamed.  Otherwise the tiles whose rounds over the CUs cost least, for experts of equal
// size (and their spread about it): a 256 x 256 tile counts 1, one of 128 x 256 0.6, one of 128 x 128 0.37.  Times in us
// of the three (128 experts, whole calls; the last two lines 8 experts):
//   rows an expert        72              96             132             200             320
//   K 4096, N 4096  486 425 425     494 431 450     504 596 650     543 709 822     911 878 1075
//   K 768, N 2048    76  70  71      90  62  65      76  83  95      87  95 113     129 125 159
//   rows an expert       100             300             700
//   K 4096, N 4096   57  48  34      78  73  73     123 115 140
//   K 1048, N 2056   42  22  19      45  25  27      41  40  43
// With fp32 sums tiles compare alike (the first line: 785 515 607, 796 518 608, 816 895 1075, 859 943 1134, 1579 1392 1660).
struct F8Plan {
    int rows, columns, group;
};
inline F8Plan f8_plan(int M, int E, int wide, int narrow, int kblocks, int num_cu) {
    const int panel = F8_PANEL / (kblocks * F8_BLOCK * 32) * 32;
    F8Plan plan;
    plan.group = panel < F8_GROUP ? panel : F8_GROUP;
    plan.rows = plan.columns = 0;
    if (M <= 64 && plan.group) return plan;
    const int64_t owners = M < E ? M : E;
    const double mean = static_cast<double>(M) / owners, most = mean + std::sqrt(mean);
    const auto cost = [&](int rows, int columns, double tile) {
        const double tiles = owners * std::ceil(most / rows) * columns;
        return std::ceil(tiles / num_cu) * tile;
    };
    plan.rows = 256;
    plan.columns = 256;
    double best = cost(256, wide, 1.0);
    if (const double c = cost(128, wide, 0.6); c < best) {
        best = c;
        plan.rows = 128;
    }
    if (narrow && cost(128, narrow, 0.37) < best) {
        plan.rows = 128;
        plan.columns = 128;
    }
    return plan;
}

// Whether a product quantizes its rows itself: all of them run as streaming items, and an expert owns few on average,
// so that every workgroup makes its own panel of them sooner than a launch of its own would.  Times in us, in the
// product and in a launch (K = N = 4096): one row for each of 8 of 128 experts 27.5, 33.4; 64 rows over 8 experts 32.4,
// 36.4; 32 rows of one expert 32.7, 23.1.
inline bool f8_quantizes(int64_t M, int64_t E, const F8Dim& k) {
    return M <= 64 && M <= 8 * (E + 1) && static_cast<int64_t>(k.padded()) * 32 <= F8_PANEL;
}

hipError_t launch_f8_quant(F8Mode mode, const F8QuantParams& p, int num_cu, hipStream_t s);
hipError_t launch_f8_gemm(F8Epilogue epilogue, const F8Params& p, int num_cu, hipStream_t s);
// w [E][n][k] in bf16 to q (e4m3) and s (a byte for each 128 x 128 block, [E][n.blocks()][k.blocks()])
hipError_t launch_f8_quant_weights(const uint16_t* w, int E, const F8Dim& n, const F8Dim& k, uint8_t* q, uint8_t* s,
                                   hipStream_t stream);
// q and s into the packed layout: the matrix is q_e, or with `transposed` q_e^T; the scales follow the matrices
hipError_t launch_f8_pack(const uint8_t* q, const uint8_t* s, int E, const F8Dim& n, const F8Dim& k, int transposed,
                          uint8_t* packed, hipStream_t stream);

}  // namespace gg
