// Internal interface between the C-ABI entry points of the expert adapters
// (gg_adapter_api.cpp) and their kernels (gg_adapter.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gg {

constexpr int AD_BLK = 32;       // rows of a block of the backward pass
constexpr int AD_WCOLS = 128;    // columns a wavefront of the backward pass owns

// Rank padded to the matrix instruction's tiles: 16, 32 or 64.
inline int ad_rank_p(int r) { return r <= 16 ? 16 : (r <= 32 ? 32 : 64); }
// Column groups (AD_WCOLS each) of a workgroup of the output-side backward
// kernel: at most (its registers hold the columns' part of db, LDS their rows), and at least;
// wavefronts that share a group, 32 ranks each; chunks of N columns.  Up to rank 16 two workgroups of
// four groups share a CU (131072 rows, Zipf, N 2048: the backward 341 us, 364 us with eight; 32768 rows, N 1536: 134 us and
// 132 us); at rank 32 the chunks' parts of du, twice as many, cost more than that gives (131072 rows: 402 us, 385 us with
// eight).
constexpr int ad_groups(int rp) { return rp == 32 ? 8 : 4; }
constexpr int ad_groups_min(int rp) { return ad_groups(rp) * 3 / 4; }
constexpr int ad_split(int rp) { return rp <= 32 ? 1 : 2; }
inline int ad_chunks(int n, int rp) { return (n + ad_groups(rp) * AD_WCOLS - 1) / (ad_groups(rp) * AD_WCOLS); }

struct AdapterParams {
    const uint16_t* x;        // [M][K]
    const int64_t* offsets;   // [E+1]
    const uint16_t* a;        // [E][r][K]
    const uint16_t* b;        // [E][N][r]
    const uint16_t* base;     // [M][N] (forward) or [M][K] (backward), or null
    int M, E, N, K, r;
    float scale;
    uint16_t* u;              // [M][r]: written by the forward, read by the backward
    uint16_t* out;            // y [M][N] or dx [M][K]
    // backward
    const uint16_t* dy;       // [M][N]
    float* da;                // [E][r][K]
    float* db;                // [E][N][r]
    int accumulate;           // da and db are added to
    int rows1, rows2;         // rows of a unit of the output-side and of the input-side kernel, about
    float* du_part;           // [chunks of N][blocks * 32][rp]: partial sums of du over the columns of a chunk
    uint16_t* du;             // [blocks][32][max(rp, 32)] bf16
    uint16_t* du_t;           // [blocks][3][rp][32] bf16: du as the sum of three parts, transposed
    float* db_part;           // [slots1][N][r]: db of the units of experts with several
    float* da_part;           // [slots2][r][K]
    int64_t blocks;           // upper bound of the row blocks
    int chunks1, chunks2;     // column chunks of the two kernels (set by the launcher)
};

hipError_t launch_adapter_forward(const AdapterParams& p, int num_cu, hipStream_t s);
hipError_t launch_adapter_backward(const AdapterParams& p, int num_cu, hipStream_t s);

}  // namespace gg
