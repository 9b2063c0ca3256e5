// Low-rank adapters of the experts on CDNA4: the forward product
// y = base + scale (x a^T) b^T and its gradients, ragged over the experts.
// The ranks are small, so every kernel is bound by the token rows it moves;
// the matrix instruction is v_mfma_f32_16x16x32_bf16 (fp32 sums).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gg_adapter.h"
#include "gg_device.h"
#include "gg_kernels.h"

namespace gg {

typedef __attribute__((ext_vector_type(4))) float f32x4;

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ bf16x8 as_bf16x8(uint4 v) { return __builtin_bit_cast(bf16x8, v); }
__device__ __forceinline__ uint4 ld16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

// Eight elements p[0], p[ld], ..., those at index >= n zero (n may be negative).
__device__ __forceinline__ uint4 gather8(const uint16_t* p, int64_t ld, int n) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) w[j >> 1] |= static_cast<uint32_t>(p[j * ld]) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------- forward
//
// A workgroup owns up to 64 rows of one expert.  U = x a^T: the four waves
// take 64-column groups of the rows in turn, each with all rows, and the
// four partial sums meet in LDS in a fixed order; U is rounded to bf16 there
// (it is saved and is the second product's operand).  Then each wave walks
// 64-column tiles of y: the tile's columns are dealt to the instruction's
// rows so that a lane ends up with 16 neighbouring columns of one token row,
// and base and y move as whole 128-byte lines without passing through LDS.
// With few row blocks the columns of y are split over workgroups, which each
// compute U again.
constexpr int AF_ROWS = 64;

template <int RP>
__global__ __launch_bounds__(256) void adapter_forward_kernel(const AdapterParams p) {
    constexpr int NT = RP / 16;                  // rank tiles
    constexpr int UW = RP < 32 ? 32 : RP;        // U's width as an operand (zero-padded)
    constexpr int KS = UW / 32;
    __shared__ int s_off[GG_KMAX_EXPERTS + 1];
    __shared__ int s_pre[GG_KMAX_EXPERTS + 1];
    __shared__ float s_part[4][AF_ROWS][RP + 4];
    __shared__ __attribute__((aligned(16))) uint16_t s_u[AF_ROWS][UW + 8];
    prefix_experts(p.offsets, p.E, p.M, s_off, s_pre, [](int m) { return (m + AF_ROWS - 1) / AF_ROWS; });
    const int blk = blockIdx.x;
    if (blk >= uni(s_pre[p.E])) return;
    const int e = uni(find_expert(s_pre, p.E, blk));
    const int row0 = uni(s_off[e]) + (blk - uni(s_pre[e])) * AF_ROWS;
    const int rows = min(AF_ROWS, uni(s_off[e + 1]) - row0);
    const int nrb = (rows + 15) / 16;
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int K = p.K, N = p.N, r = p.r;
    const uint16_t* ae = p.a + static_cast<int64_t>(e) * r * K;
    const uint16_t* be = p.b + static_cast<int64_t>(e) * N * r;

    // ---- U
    {
        const uint16_t* xr[4];
        const uint16_t* ar[NT];
#pragma unroll
        for (int i = 0; i < 4; ++i) xr[i] = p.x + static_cast<int64_t>(row0 + min(16 * i + l16, rows - 1)) * K;
#pragma unroll
        for (int j = 0; j < NT; ++j) ar[j] = ae + static_cast<int64_t>(min(16 * j + l16, r - 1)) * K;
        f32x4 acc[4][NT];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
        uint4 xv[2][2][4], av[2][2][NT];
        const int groups = (K + 63) / 64;
        auto load = [&](int buf, int grp) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int k = grp * 64 + c * 32 + 8 * g;
                const bool in = k < K;
                const int kc = in ? k : 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < nrb) xv[buf][c][i] = ld16(xr[i] + kc);
#pragma unroll
                for (int j = 0; j < NT; ++j) av[buf][c][j] = ld16(ar[j] + kc);
                if (grp * 64 + 64 > K) {   // past the end both operands are zero
                    const uint32_t keep = in ? ~0u : 0u;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        xv[buf][c][i] = make_uint4(xv[buf][c][i].x & keep, xv[buf][c][i].y & keep, xv[buf][c][i].z & keep,
                                                   xv[buf][c][i].w & keep);
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        av[buf][c][j] = make_uint4(av[buf][c][j].x & keep, av[buf][c][j].y & keep, av[buf][c][j].z & keep,
                                                   av[buf][c][j].w & keep);
                }
            }
        };
        auto mma = [&](int buf) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < nrb) {
#pragma unroll
                        for (int j = 0; j < NT; ++j)
                            acc[i][j] = mfma16(as_bf16x8(av[buf][c][j]), as_bf16x8(xv[buf][c][i]), acc[i][j]);
                    }
        };
        int grp = wave;
        if (grp < groups) load(0, grp);
        for (; grp < groups; grp += 8) {
            if (grp + 4 < groups) load(1, grp + 4);
            mma(0);
            if (grp + 4 < groups) {
                if (grp + 8 < groups) load(0, grp + 8);
                mma(1);
            }
        }
        // lane: row 16 i + l16, ranks 16 j + 4 g ..
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (i < nrb) *reinterpret_cast<f32x4*>(&s_part[wave][16 * i + l16][16 * j + 4 * g]) = acc[i][j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < AF_ROWS * UW; i += 256) {
        const int row = i / UW, c = i % UW;
        float v = 0.0f;
        if (row < rows && c < r)
            v = (s_part[0][row][c] + s_part[1][row][c]) + (s_part[2][row][c] + s_part[3][row][c]);
        const uint16_t h = f2bf(v);
        s_u[row][c] = h;
        if (row < rows && c < r && blockIdx.y == 0) p.u[static_cast<int64_t>(row0 + row) * r + c] = h;
    }
    __syncthreads();

    // ---- y
    bf16x8 uo[4][KS];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < KS; ++k) uo[i][k] = *reinterpret_cast<const bf16x8*>(&s_u[16 * i + l16][32 * k + 8 * g]);
    const bool r8 = (r & 7) == 0;
    const int tiles = (N + 63) / 64;
    const int per = (tiles + gridDim.y - 1) / gridDim.y;
    const int t1 = min(tiles, static_cast<int>(blockIdx.y + 1) * per);
    for (int ct = blockIdx.y * per + wave; ct < t1; ct += 4) {
        const int n0 = ct * 64 + 16 * g;            // the lane's 16 columns
        uint4 bv[4][KS], base[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                base[i][h] = make_uint4(0, 0, 0, 0);
                if (p.base && 16 * i + l16 < rows && n0 + 8 * h < N)
                    base[i][h] = ld16(p.base + static_cast<int64_t>(row0 + 16 * i + l16) * N + n0 + 8 * h);
            }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int c = min(ct * 64 + 16 * (l16 >> 2) + 4 * t + (l16 & 3), N - 1);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int c0 = 32 * k + 8 * g;
                const uint16_t* src = be + static_cast<int64_t>(c) * r + c0;
                if (r8) bv[t][k] = c0 < r ? ld16(src) : make_uint4(0, 0, 0, 0);
                else bv[t][k] = gather8(src, 1, r - c0);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= nrb) continue;
            f32x4 d[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                d[t] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KS; ++k) d[t] = mfma16(as_bf16x8(bv[t][k]), uo[i][k], d[t]);
            }
            if (16 * i + l16 >= rows) continue;
            uint16_t* yrow = p.out + static_cast<int64_t>(row0 + 16 * i + l16) * N + n0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (n0 + 8 * h >= N) continue;
                const uint32_t bw[4] = {base[i][h].x, base[i][h].y, base[i][h].z, base[i][h].w};
                uint32_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4& dd = d[2 * h + (q >> 1)];
                    o[q] = pack2(lo_f(bw[q]) + p.scale * dd[2 * (q & 1)], hi_f(bw[q]) + p.scale * dd[2 * (q & 1) + 1]);
                }
                *reinterpret_cast<uint4*>(yrow + 8 * h) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

// ---------------------------------------------------------------- backward
//
// Four launches over 32-row blocks that start at each expert's first row:
//   1  output side: a unit is up to rows1 rows of one expert x a chunk of dy's
//      columns.  It reads dy once and makes both products of it: db (summed
//      over the rows in registers) and the chunk's part of du = scale dy b.
//   2  du: the chunks' parts added in order, rounded to bf16 for dx, and kept
//      whole as the sum of three bf16 values for da, whose output is fp32.
//   3  input side: a unit is up to rows2 rows of one expert x 512 columns of x:
//      da (summed in registers) and dx = base + du a.
//   4  experts with several units: their parts added in order; experts without
//      rows: zeros.
// A sum over rows needs the rows as the instruction's summed dimension: a lane
// loads the same 8 columns of 8 rows (256-byte row segments across 16 lanes)
// and pairs them up by byte permutes, so its 8 operands are 8 columns with 8
// rows each.
__device__ __forceinline__ void transpose8(const uint4 (&in)[8], uint4 (&out)[8]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t a[4] = {in[2 * q].x, in[2 * q].y, in[2 * q].z, in[2 * q].w};
            const uint32_t b[4] = {in[2 * q + 1].x, in[2 * q + 1].y, in[2 * q + 1].z, in[2 * q + 1].w};
            lo[q] = __builtin_amdgcn_perm(b[c], a[c], 0x05040100u);
            hi[q] = __builtin_amdgcn_perm(b[c], a[c], 0x07060302u);
        }
        out[2 * c] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        out[2 * c + 1] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
}

// One unit of work: rows [row0, row0 + rows) of expert e, its first 32-row
// block blk0, and its slot among the parts of experts with several units (-1: its expert has one).
struct AdapterUnit {
    int e, row0, rows, blk0, slot;
};

// The schedule in LDS: units, 32-row blocks and part slots before each expert.
struct AdapterSchedule {
    int off[GG_KMAX_EXPERTS + 1], unit[GG_KMAX_EXPERTS + 1], blk[GG_KMAX_EXPERTS + 1], slot[GG_KMAX_EXPERTS + 1];
};

__device__ __forceinline__ void build_units(const AdapterParams& p, int unit_rows, AdapterSchedule& s) {
    prefix_experts(p.offsets, p.E, p.M, s.off, s.unit, [&](int m) { return (m + unit_rows - 1) / unit_rows; });
    prefix_experts(p.offsets, p.E, p.M, s.off, s.blk, [&](int m) { return (m + AD_BLK - 1) / AD_BLK; });
    prefix_experts(p.offsets, p.E, p.M, s.off, s.slot,
                   [&](int m) { return m > unit_rows ? (m + unit_rows - 1) / unit_rows : 0; });
}

__device__ __forceinline__ AdapterUnit unit_at(const AdapterParams& p, int unit_rows, const AdapterSchedule& s, int i) {
    AdapterUnit u;
    u.e = uni(find_expert(s.unit, p.E, i));
    const int part = i - uni(s.unit[u.e]);
    const int lo = uni(s.off[u.e]), hi = uni(s.off[u.e + 1]);
    u.row0 = lo + part * unit_rows;
    u.rows = min(unit_rows, hi - u.row0);
    u.blk0 = uni(s.blk[u.e]) + part * (unit_rows / AD_BLK);
    u.slot = hi - lo > unit_rows ? uni(s.slot[u.e]) + part : -1;
    return u;
}

// Eight rows 8 g + t of the 32-row block at `row`, columns c .. c+7 (`in`: those exist); rows past `rows` are zero.
__device__ __forceinline__ void load_rows8(const uint16_t* m, int64_t ld, int row0, int row, int rows, int c, bool in,
                                           uint4 (&v)[8]) {
    const int g = (threadIdx.x & 63) >> 4;
    const uint16_t* base = m + static_cast<int64_t>(row0) * ld + (in ? c : 0);
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = ld16(base + static_cast<int64_t>(min(row + 8 * g + t, rows - 1)) * ld);
}
__device__ __forceinline__ void mask_rows8(int row, int rows, bool in, uint4 (&v)[8]) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const uint32_t keep = in && row + 8 * g + t < rows ? ~0u : 0u;
        v[t] = make_uint4(v[t].x & keep, v[t].y & keep, v[t].z & keep, v[t].w & keep);
    }
}

template <int RP>
__global__ __launch_bounds__(RP <= 32 ? 512 : 256) void adapter_dy_kernel(const AdapterParams p) {
    constexpr int NW = RP <= 32 ? 8 : 4;
    constexpr int NT = RP / 16;
    __shared__ AdapterSchedule s;
    // each wave's 32 x 128 tile of dy; 16-byte chunk c of row i at c ^ (i & 15)
    __shared__ __attribute__((aligned(16))) uint16_t s_dy[NW][AD_BLK * AD_WCOLS];
    __shared__ __attribute__((aligned(16))) uint16_t s_ut[2][RP][AD_BLK + 8];    // U^T of a block
    __shared__ float s_du[2][NW][AD_BLK][RP + 4];                                // the waves' parts of du
    build_units(p, p.rows1, s);
    if (static_cast<int>(blockIdx.x) >= uni(s.unit[p.E])) return;
    const AdapterUnit un = unit_at(p, p.rows1, s, blockIdx.x);
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int N = p.N, r = p.r;
    const int c0 = (blockIdx.y * NW + wave) * AD_WCOLS;
    const int cl = c0 + 8 * l16;                  // the lane's columns
    const bool in = cl < N;
    const bool whole = c0 + AD_WCOLS <= N;
    const uint16_t* be = p.b + static_cast<int64_t>(un.e) * N * r;
    const uint16_t* ue = p.u + static_cast<int64_t>(un.row0) * r;

    bf16x8 bw[4][NT];   // b as the operand of du: rank 16 j + l16, columns c0 + 32 k + 8 g ..
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int c = c0 + 32 * k + 8 * g, rr = 16 * j + l16;
            bw[k][j] = as_bf16x8(gather8(be + static_cast<int64_t>(c) * r + rr, r, rr < r ? N - c : 0));
        }
    f32x4 acc[8][NT];
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[c][j] = f32x4{0, 0, 0, 0};

    constexpr int UPT = AD_BLK * RP / (NW * 64);   // U elements a thread stages
    uint16_t uv[UPT];
    auto load_u = [&](int row) {
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const int el = tid + i * NW * 64, rr = el / RP, c = el % RP;
            uv[i] = row + rr < un.rows && c < r ? ue[static_cast<int64_t>(row + rr) * r + c] : 0;
        }
    };
    auto put_u = [&](int buf) {
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const int el = tid + i * NW * 64;
            s_ut[buf][el % RP][el / RP] = uv[i];
        }
    };
    uint4 cur[8], nxt[8];
    load_rows8(p.dy, N, un.row0, 0, un.rows, cl, in, cur);
    load_u(0);
    put_u(0);
    __syncthreads();
    int buf = 0;
    for (int row = 0; row < un.rows; row += AD_BLK, buf ^= 1) {
        const bool more = row + AD_BLK < un.rows;
        if (more) {
            load_rows8(p.dy, N, un.row0, row + AD_BLK, un.rows, cl, in, nxt);
            load_u(row + AD_BLK);
        }
        if (!whole || row + AD_BLK > un.rows) mask_rows8(row, un.rows, in, cur);
        uint16_t* tile = s_dy[wave];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int rr = 8 * g + t;
            *reinterpret_cast<uint4*>(tile + rr * AD_WCOLS + ((l16 ^ (rr & 15)) << 3)) = cur[t];
        }
        uint4 tr[8];
        transpose8(cur, tr);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const bf16x8 ut = *reinterpret_cast<const bf16x8*>(&s_ut[buf][16 * j + l16][8 * g]);
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[c][j] = mfma16(as_bf16x8(tr[c]), ut, acc[c][j]);
        }
        f32x4 du[2][NT];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NT; ++j) du[h][j] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int rr = 16 * h + l16;
                const bf16x8 d = *reinterpret_cast<const bf16x8*>(tile + rr * AD_WCOLS + (((4 * k + g) ^ (rr & 15)) << 3));
#pragma unroll
                for (int j = 0; j < NT; ++j) du[h][j] = mfma16(bw[k][j], d, du[h][j]);
            }
        // lane: row 16 h + l16, ranks 16 j + 4 g ..
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                *reinterpret_cast<f32x4*>(&s_du[buf][wave][16 * h + l16][16 * j + 4 * g]) = du[h][j];
        if (more) put_u(buf ^ 1);
        __syncthreads();   // the waves' parts are in; the next block's go to the other buffers
        float* part = p.du_part + ((static_cast<int64_t>(blockIdx.y) * p.blocks + un.blk0 + row / AD_BLK) * AD_BLK) * RP;
        for (int i = tid; i < AD_BLK * RP / 4; i += NW * 64) {
            const int rr = i / (RP / 4), c = i % (RP / 4) * 4;
            f32x4 sum = *reinterpret_cast<const f32x4*>(&s_du[buf][0][rr][c]);
#pragma unroll
            for (int w = 1; w < NW; ++w) sum += *reinterpret_cast<const f32x4*>(&s_du[buf][w][rr][c]);
            *reinterpret_cast<f32x4*>(part + rr * RP + c) = sum;
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) cur[t] = nxt[t];
    }
    // lane: rank 16 j + l16, columns c0 + 8 (4 g + x) + c
    const bool direct = un.slot < 0;
    float* out = direct ? p.db + static_cast<int64_t>(un.e) * N * r : p.db_part + static_cast<int64_t>(un.slot) * N * r;
    const bool add = direct && p.accumulate;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int n = c0 + 8 * (4 * g + x) + c, rr = 16 * j + l16;
                if (n < N && rr < r) {
                    float* o = out + static_cast<int64_t>(n) * r + rr;
                    const float v = p.scale * acc[c][j][x];
                    *o = add ? *o + v : v;
                }
            }
}

// du of every block from its parts, in chunk order; rows past an expert's end are zero already.
template <int RP>
__global__ __launch_bounds__(256) void adapter_du_kernel(const AdapterParams p, int chunks) {
    constexpr int UW = RP < 32 ? 32 : RP;
    __shared__ int s_off[GG_KMAX_EXPERTS + 1];
    __shared__ int s_blk[GG_KMAX_EXPERTS + 1];
    prefix_experts(p.offsets, p.E, p.M, s_off, s_blk, [](int m) { return (m + AD_BLK - 1) / AD_BLK; });
    const int64_t total = static_cast<int64_t>(uni(s_blk[p.E])) * AD_BLK * RP;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        // consecutive threads take consecutive rows of one rank, so that the transposed stores are contiguous
        const int64_t blk = i / (AD_BLK * RP);
        const int w = static_cast<int>(i % (AD_BLK * RP)), c = w / AD_BLK, row = w % AD_BLK;
        const float* src = p.du_part + (blk * AD_BLK + row) * RP + c;
        float v = 0.0f;
        for (int k = 0; k < chunks; ++k) v += src[static_cast<int64_t>(k) * p.blocks * AD_BLK * RP];
        v *= p.scale;
        const uint16_t hi = f2bf(v);
        const float rest = v - bf2f(hi);
        const uint16_t mid = f2bf(rest), lo = f2bf(rest - bf2f(mid));
        p.du[(blk * AD_BLK + row) * UW + c] = hi;
        if (RP < UW) p.du[(blk * AD_BLK + row) * UW + RP + c] = 0;
        uint16_t* t = p.du_t + (blk * 3 * RP + c) * AD_BLK + row;
        t[0] = hi;
        t[RP * AD_BLK] = mid;
        t[2 * RP * AD_BLK] = lo;
    }
}

template <int RP>
__global__ __launch_bounds__(256) void adapter_dx_kernel(const AdapterParams p) {
    constexpr int NT = RP / 16;
    constexpr int UW = RP < 32 ? 32 : RP;
    constexpr int KS = UW / 32;
    __shared__ AdapterSchedule s;
    build_units(p, p.rows2, s);
    if (static_cast<int>(blockIdx.x) >= uni(s.unit[p.E])) return;
    const AdapterUnit un = unit_at(p, p.rows2, s, blockIdx.x);
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int K = p.K, r = p.r;
    const int c0 = (blockIdx.y * 4 + wave) * AD_WCOLS;
    if (c0 >= K) return;
    const int cl = c0 + 8 * l16;
    const bool in = cl < K, whole = c0 + AD_WCOLS <= K;
    const uint16_t* ae = p.a + static_cast<int64_t>(un.e) * r * K;

    // a as the operand of dx: tile t of 64-column half h, ranks 32 k + 8 g ..
    bf16x8 aw[2][4][KS];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int c = c0 + 64 * h + 16 * (l16 >> 2) + 4 * t + (l16 & 3), rr = 32 * k + 8 * g;
                aw[h][t][k] = as_bf16x8(gather8(ae + static_cast<int64_t>(rr) * K + c, K, c < K ? r - rr : 0));
            }
    f32x4 acc[8][NT];
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[c][j] = f32x4{0, 0, 0, 0};
    uint4 cur[8], nxt[8];
    load_rows8(p.x, K, un.row0, 0, un.rows, cl, in, cur);
    for (int row = 0; row < un.rows; row += AD_BLK) {
        const int64_t blk = un.blk0 + row / AD_BLK;
        uint4 base[2][2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int rr = row + 16 * i + l16, c = c0 + 64 * h + 16 * g + 8 * q;
                    base[i][h][q] = make_uint4(0, 0, 0, 0);
                    if (p.base && rr < un.rows && c < K)
                        base[i][h][q] = ld16(p.base + static_cast<int64_t>(un.row0 + rr) * K + c);
                }
        bf16x8 dt[3][NT], dr[2][KS];
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                dt[q][j] = as_bf16x8(ld16(p.du_t + ((blk * 3 + q) * RP + 16 * j + l16) * AD_BLK + 8 * g));
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < KS; ++k)
                dr[i][k] = as_bf16x8(ld16(p.du + (blk * AD_BLK + 16 * i + l16) * UW + 32 * k + 8 * g));
        if (row + AD_BLK < un.rows) load_rows8(p.x, K, un.row0, row + AD_BLK, un.rows, cl, in, nxt);
        if (!whole || row + AD_BLK > un.rows) mask_rows8(row, un.rows, in, cur);
        uint4 tr[8];
        transpose8(cur, tr);
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int q = 2; q >= 0; --q) acc[c][j] = mfma16(as_bf16x8(tr[c]), dt[q][j], acc[c][j]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x4 d[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    d[t] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < KS; ++k) d[t] = mfma16(aw[h][t][k], dr[i][k], d[t]);
                }
                const int rr = row + 16 * i + l16;
                if (rr >= un.rows) continue;
                uint16_t* orow = p.out + static_cast<int64_t>(un.row0 + rr) * K + c0 + 64 * h + 16 * g;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (c0 + 64 * h + 16 * g + 8 * q >= K) continue;
                    const uint32_t bw[4] = {base[i][h][q].x, base[i][h][q].y, base[i][h][q].z, base[i][h][q].w};
                    uint32_t o[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const f32x4& dd = d[2 * q + (m >> 1)];
                        o[m] = pack2(lo_f(bw[m]) + dd[2 * (m & 1)], hi_f(bw[m]) + dd[2 * (m & 1) + 1]);
                    }
                    *reinterpret_cast<uint4*>(orow + 8 * q) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
#pragma unroll
        for (int t = 0; t < 8; ++t) cur[t] = nxt[t];
    }
    // lane: rank 16 j + l16, columns c0 + 8 (4 g + x) + 0 .. 7
    const bool direct = un.slot < 0;
    float* out = direct ? p.da + static_cast<int64_t>(un.e) * r * K : p.da_part + static_cast<int64_t>(un.slot) * r * K;
    const bool add = direct && p.accumulate;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int c = c0 + 8 * (4 * g + x), rr = 16 * j + l16;
            if (c >= K || rr >= r) continue;
            float* o = out + static_cast<int64_t>(rr) * K + c;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x4 v = {acc[4 * h][j][x], acc[4 * h + 1][j][x], acc[4 * h + 2][j][x], acc[4 * h + 3][j][x]};
                if (add) v += *reinterpret_cast<const f32x4*>(o + 4 * h);
                *reinterpret_cast<f32x4*>(o + 4 * h) = v;
            }
        }
}

// Experts with several units: the parts in order; experts without rows: zeros
// (unless the gradients accumulate).  A workgroup serves one expert;
// blockIdx.y: 0 for db, 1 for da.
__global__ __launch_bounds__(256) void adapter_join_kernel(const AdapterParams p) {
    __shared__ int s_off[GG_KMAX_EXPERTS + 1];
    __shared__ int s_slot[GG_KMAX_EXPERTS + 1];
    const int unit_rows = blockIdx.y ? p.rows2 : p.rows1;
    const int e = blockIdx.z;
    auto clamped = [&](int i) {
        const int64_t o = p.offsets[i];
        return static_cast<int>(o < 0 ? 0 : (o > p.M ? p.M : o));
    };
    const int m = uni(clamped(e + 1) - clamped(e));
    if (m > 0 ? m <= unit_rows : p.accumulate) return;   // written by its one unit, or nothing to add
    int s0 = 0, n = 0;
    if (m > 0) {
        prefix_experts(p.offsets, p.E, p.M, s_off, s_slot,
                       [&](int m) { return m > unit_rows ? (m + unit_rows - 1) / unit_rows : 0; });
        s0 = uni(s_slot[e]);
        n = uni(s_slot[e + 1]) - s0;
    }
    const int64_t size = static_cast<int64_t>(p.r) * (blockIdx.y ? p.K : p.N);   // a multiple of 4
    const float* part = blockIdx.y ? p.da_part : p.db_part;
    float* out = (blockIdx.y ? p.da : p.db) + e * size;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < size;
         i += static_cast<int64_t>(gridDim.x) * 1024) {
        f32x4 v = {0, 0, 0, 0};
        for (int k = 0; k < n; ++k) v += *reinterpret_cast<const f32x4*>(part + (s0 + k) * size + i);
        f32x4* o = reinterpret_cast<f32x4*>(out + i);
        if (p.accumulate) v += *o;
        *o = v;
    }
}

// ---------------------------------------------------------------- launchers
template <int RP>
static hipError_t forward_of(const AdapterParams& p, int num_cu, hipStream_t s) {
    const int64_t blocks = static_cast<int64_t>(p.M) / AF_ROWS + (p.M < p.E ? p.M : p.E);
    // two workgroups for each CU where the rows alone give fewer, down to 256 columns each
    int64_t split = 2 * static_cast<int64_t>(num_cu) / blocks;
    const int64_t most = (p.N + 255) / 256;
    split = split < 1 ? 1 : (split > most ? most : split);
    hipLaunchKernelGGL((adapter_forward_kernel<RP>), dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(split)),
                       dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_adapter_forward(const AdapterParams& p, int num_cu, hipStream_t s) {
    switch (ad_rank_p(p.r)) {
        case 16: return forward_of<16>(p, num_cu, s);
        case 32: return forward_of<32>(p, num_cu, s);
        default: return forward_of<64>(p, num_cu, s);
    }
}

template <int RP>
static hipError_t backward_of(const AdapterParams& p, int num_cu, hipStream_t s) {
    const int64_t few = p.M < p.E ? p.M : p.E;
    const int cols = ad_waves(RP) * AD_WCOLS;
    const int chunks = (p.N + cols - 1) / cols;
    hipError_t st;
    if (p.M > 0) {
        hipLaunchKernelGGL((adapter_dy_kernel<RP>),
                           dim3(static_cast<unsigned>(p.M / p.rows1 + few), static_cast<unsigned>(chunks)),
                           dim3(ad_waves(RP) * 64), 0, s, p);
        if ((st = hipGetLastError()) != hipSuccess) return st;
        const int64_t want = p.blocks * AD_BLK * RP / 256, most = static_cast<int64_t>(num_cu) * 8;
        hipLaunchKernelGGL((adapter_du_kernel<RP>), dim3(static_cast<unsigned>(want < most ? want : most)), dim3(256), 0, s, p,
                           chunks);
        if ((st = hipGetLastError()) != hipSuccess) return st;
        hipLaunchKernelGGL((adapter_dx_kernel<RP>),
                           dim3(static_cast<unsigned>(p.M / p.rows2 + few), static_cast<unsigned>((p.K + 511) / 512)), dim3(256),
                           0, s, p);
        if ((st = hipGetLastError()) != hipSuccess) return st;
    }
    const int64_t width = p.N > p.K ? p.N : p.K, gx = (width * p.r / 4 + 1023) / 1024;
    hipLaunchKernelGGL(adapter_join_kernel, dim3(static_cast<unsigned>(gx < 16 ? gx : 16), 2, static_cast<unsigned>(p.E)),
                       dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_adapter_backward(const AdapterParams& p, int num_cu, hipStream_t s) {
    switch (ad_rank_p(p.r)) {
        case 16: return backward_of<16>(p, num_cu, s);
        case 32: return backward_of<32>(p, num_cu, s);
        default: return backward_of<64>(p, num_cu, s);
    }
}

}  // namespace gg
