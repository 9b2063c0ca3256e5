// Internal interface between the C-ABI entry points of the 8-bit expert
// products (gg_int8_api.cpp) and their kernels (gg_int8.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gg {

// Layout of a packed 8-bit matrix W [rows][cont] (rows: output columns of the
// product, cont: the summed dimension): 32-row blocks, each of cont_p / 32
// steps of 1 KiB in the operand order of the 32x32x32 int8 matrix
// instruction: lane l's 16 bytes are row 32b + (l & 31), columns
// 32s + 16(l >> 5) onwards.  Both dimensions are padded with zeros.
constexpr int I8_ROWS = 32, I8_STEP = 32, I8_PAD = 128;
inline int64_t i8_rows_p(int64_t rows) { return (rows + I8_ROWS - 1) / I8_ROWS * I8_ROWS; }
inline int64_t i8_cont_p(int64_t cont) { return (cont + I8_PAD - 1) / I8_PAD * I8_PAD; }

// What a row's 8-bit values are made from.
enum QuantMode {
    Q_PLAIN = 0,    // v = x
    Q_GLU = 1,      // v = bf16(act(gate) * up) of x = [gate | up]
    Q_SCALED = 2,   // v = cs_e[n] * x[n]
    Q_DGLU = 3      // v = cs_e[n] * dH1[n], dH1 = bf16(derivative of the activation at h1, times x)
};

struct QuantParams {
    const uint16_t* x;       // [M][K] bf16 (Q_GLU: [M][2K], Q_DGLU: [M][K/2])
    const uint16_t* h1;      // Q_DGLU: [M][K]
    const int64_t* offsets;  // [E+1], or null: every row below M
    const float* cs;         // Q_SCALED, Q_DGLU: column scales [E][cs_ld]
    int cs_ld;
    int M, E, K;             // K: values of a quantized row
    float slope;
    uint16_t* v_out;         // Q_GLU: A [M][K], Q_DGLU: dH1 [M][K]; null: not kept
    int8_t* q;               // column c of row r at (c / 64) * q_block + r * q_row + c % 64
    int64_t q_block, q_row;  // (64, K): rows as they are; (64 M, 64): blocks of 64 columns, for the product
    int blocked;             // the latter
    int width;               // columns written: K, or K padded with zeros
    float* s;                // [M]
};

// out[r][n] = bf16(s[r] * ws_e[n] * sum_k q[r][k] W_e[n][k])
struct Int8Params {
    const int8_t* q;         // [width / 64][M][64]
    const float* s;          // [M]
    const int64_t* offsets;  // [E+1]
    const int8_t* w;         // packed matrices
    int64_t w_stride;        // bytes of one expert's matrix
    const float* ws;         // [E][ws_ld] output column scales, or null (all one)
    int ws_ld;
    int width;               // summed dimension, padded (a multiple of 128)
    int M, E, N;             // N: output columns, a multiple of 8
    uint16_t* out;           // [M][N]
    int tile;                // rows of a tile, or 0: no tiles (set by the launcher)
    int group;               // rows of a streaming item, at most; 0: this launch has none (set by the launcher)
};

constexpr int I8_GROUP = 96;          // rows of a streaming item, at most
constexpr int I8_RING = 128 * 1024;   // LDS for operands

// Which tiles a product of M rows over E experts, N columns and a summed width takes (rows of a tile, 0: none), and
// how many rows a streaming item in the tiles' launch has at most (0: the streaming items have a launch of their own).
//
// No expert of a batch of few rows has a tile.  Small tiles where the rows would make fewer large ones than
// CUs (8 experts of 300 rows, K 1048, N 2056: 28 us, 44 us with large ones), and from 80 to 119 rows an expert on average: such experts fill a small tile, and less than half of a large
// one, or stream.  Times in us, small and large tiles, 128 experts, uniform:
//   rows an expert          64         72         80         96        116        132        200
//   K 4096, N 4096     650  702   516  738   490  821   475  670   506  563   664  557   890  629
//   K 2688, N 3712     405  406   338  433   318  472   317  444   339  376   427  379   561  429
//   K 768, N 2048       77   63    82   65    82   83    75   90    84   93   109   88   137   99
// Below, 36 rows: 413 and 329 (K 2688, N 3712: LDS holds 32 rows, so small tiles' launch reads the weights of 33
// twice).  Zipf-distributed experts of 72 to 120 rows on average: within 7% of each other either way.
//
// Tiles and the rows they leave share a launch where LDS holds 32 rows of the summed width, or, of what large
// tiles leave, 64, so that few weights are read twice (128 experts of 300 rows, K 2048, N 1536: 245 us, 267 us in
// two launches).
struct Int8Plan {
    int tile, group;
};
inline Int8Plan i8_plan(int M, int E, int N, int width, int num_cu) {
    const int64_t large = static_cast<int64_t>(M) / 256 * ((N + 255) / 256);
    const int64_t owners = M < E ? M : E;
    const bool half = M >= 80 * owners && M < 120 * owners;
    Int8Plan plan;
    plan.tile = M <= 64 ? 0 : (large < num_cu || half ? 128 : 256);
    const int panel = I8_RING / (width * 32) * 32, least = plan.tile == 256 ? 64 : 32;
    plan.group = plan.tile == 0 || panel < least ? 0 : (panel < I8_GROUP ? panel : I8_GROUP);
    return plan;
}

// How a wave of the quantization takes Y (1 or 2) rows of [lo, hi) at a time: from i8_first_row, in steps of Y, while
// below hi.  Pairs start at an even row, so that the two rows share their lines; a pair of which one row lies
// outside holds its other row twice.  No rows (lo >= hi): no step at all, also where lo is odd.
template <int Y>
__host__ __device__ inline int i8_first_row(int lo, int hi) {
    return Y == 2 && lo < hi ? lo & ~1 : lo;
}
template <int Y>
__host__ __device__ inline void i8_rows_at(int64_t r0, int lo, int hi, int64_t (&row)[Y]) {
    row[0] = r0 < lo ? r0 + 1 : r0;
    if (Y == 2) row[Y - 1] = r0 + 1 < hi ? r0 + 1 : r0;
}

hipError_t launch_quant_rows(QuantMode mode, const QuantParams& p, int num_cu, hipStream_t s);
hipError_t launch_int8_gemm(const Int8Params& p, int num_cu, hipStream_t s);
// q [E][N][K] and s [E][N] into the packed layout: W = q_e (rows N, summed K), or with
// `transposed` q_e^T (rows K, summed N); the scales [E][i8_cont_p(N)] follow the matrices.
hipError_t launch_int8_pack(const int8_t* q, const float* s, int E, int N, int K, int transposed, int8_t* packed,
                            hipStream_t stream);

}  // namespace gg
