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

// Eight elements p[0], p[ld], ..., of which the first n exist (p[0] is
// readable in any case); the others are zero.  All eight loads are issued
// without a branch between them.
__device__ __forceinline__ uint4 gather8(const uint16_t* p, int64_t ld, int n) {
    uint32_t v[8];
    const int top = max(n - 1, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = p[min(j, top) * ld];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j >= n) v[j] = 0;
    return make_uint4(v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16), v[6] | (v[7] << 16));
}

// ---------------------------------------------------------------- forward
//
// A workgroup owns up to 16 RB rows of one expert, as 16-row blocks (RB = 4,
// or 2 with twice the waves where the experts have few rows).  U = x a^T: the
// waves take 64-column groups of the rows in turn, each with all rows, and
// their partial sums meet in LDS in a fixed order; U is rounded to bf16 there,
// once: what is saved is what y is made of, so that db = dy^T u is y's own gradient.
// y is bf16 itself; with u whole its relative error (root mean square, base and
// update of normals) would be 0.00166 for 0.00171, without a base 0.00166 for 0.00234.
// Then each wave walks 128-column tiles of y: the columns are dealt to the
// eight instructions of a tile so that a lane ends up with 8 neighbouring
// columns of four token rows, and base and y move as 256-byte row segments of
// 16 lanes without passing through LDS.  With few row blocks the columns of y
// are split over workgroups, which each compute U again.
// Bound by HBM in large batches (262144 rows, K = N = 4096, rank 32: 1.30 ms, 5.6
// TB/s), by the chain offsets - x and a - b in small ones (one token's 8
// rows: 10 us; 2880 rows over 128 experts, K 2688, N 3712, rank 12: 31 us, 2.5 TB/s).
constexpr int af_waves(int rb) { return rb == 2 ? 8 : 4; }

__device__ __forceinline__ uint4 and4(uint4 v, uint32_t m) { return make_uint4(v.x & m, v.y & m, v.z & m, v.w & m); }

// This wave's part of U for the NRB 16-row blocks from row0: groups wave,
// wave + W, ... of 64 columns, D of them loaded ahead while D are multiplied.
// Lane: row 16 i + (lane & 15), ranks 16 j + 4 (lane >> 4) .. of acc[i][j].
template <int NT, int NRB, int D, int W, int MAXB>
__device__ __forceinline__ void adapter_u(const AdapterParams& p, const uint16_t* ae, int row0, int rows, int wave,
                                          f32x4 (&acc)[MAXB][NT]) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
    const int K = p.K, groups = (K + 63) / 64;
    const uint16_t* xr[NRB];
    const uint16_t* ar[NT];
#pragma unroll
    for (int i = 0; i < NRB; ++i) xr[i] = p.x + static_cast<int64_t>(row0 + min(16 * i + l16, rows - 1)) * K;
#pragma unroll
    for (int j = 0; j < NT; ++j) ar[j] = ae + static_cast<int64_t>(min(16 * j + l16, p.r - 1)) * K;
    uint4 xv[2][D][2][NRB], av[2][D][2][NT];
    // groups first, first + W, ...; past the end of the columns both operands are zero
    auto load = [&](int buf, int first) {
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int k = (first + W * d) * 64 + c * 32 + 8 * g;
                const int kc = k < K ? k : 0;
#pragma unroll
                for (int i = 0; i < NRB; ++i) xv[buf][d][c][i] = ld16(xr[i] + kc);
#pragma unroll
                for (int j = 0; j < NT; ++j) av[buf][d][c][j] = ld16(ar[j] + kc);
            }
    };
    auto mma = [&](int buf, int first) {
        if ((first + W * (D - 1) + 1) * 64 > K) {
#pragma unroll
            for (int d = 0; d < D; ++d)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t keep = (first + W * d) * 64 + c * 32 + 8 * g < K ? ~0u : 0u;
#pragma unroll
                    for (int i = 0; i < NRB; ++i) xv[buf][d][c][i] = and4(xv[buf][d][c][i], keep);
#pragma unroll
                    for (int j = 0; j < NT; ++j) av[buf][d][c][j] = and4(av[buf][d][c][j], keep);
                }
        }
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < NRB; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[i][j] = mfma16(as_bf16x8(av[buf][d][c][j]), as_bf16x8(xv[buf][d][c][i]), acc[i][j]);
    };
    int at = wave;
    if (at < groups) load(0, at);
    for (; at < groups; at += 2 * W * D) {
        if (at + W * D < groups) load(1, at + W * D);
        mma(0, at);
        if (at + W * D < groups) {
            if (at + 2 * W * D < groups) load(0, at + 2 * W * D);
            mma(1, at + W * D);
        }
    }
}

template <int RP, int RB>
__global__ __launch_bounds__(af_waves(RB) * 64, 2) void adapter_forward_kernel(const AdapterParams p) {
    constexpr int W = af_waves(RB), AF_ROWS = 16 * RB;
    constexpr int NT = RP / 16;                  // rank tiles
    constexpr int UW = RP < 32 ? 32 : RP;        // U's width as an operand (zero-padded)
    constexpr int KS = UW / 32;
    __shared__ __attribute__((aligned(16))) float s_part[W][AF_ROWS][RP + 4];
    __shared__ __attribute__((aligned(16))) uint16_t s_u[AF_ROWS][UW + 8];
    const ExpertItem<1> it = find_item<1>(p.offsets, p.E, p.M, blockIdx.x,
                                          [](int m) { return Counts<1>{{(m + AF_ROWS - 1) / AF_ROWS}}; });
    if (it.e < 0) return;
    const int e = it.e;
    const int row0 = it.lo + (static_cast<int>(blockIdx.x) - it.before[0]) * AF_ROWS;
    const int rows = min(AF_ROWS, it.hi - row0);
    const int nrb = (rows + 15) / 16;
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int N = p.N, r = p.r;
    const uint16_t* ae = p.a + static_cast<int64_t>(e) * r * p.K;

    // b's rows are 2 r bytes apart: a 16-byte load may start anywhere and may reach into the next
    // row, whose values are cleared, but not past the tensor's end
    const uint16_t* be = p.b + static_cast<int64_t>(e) * N * r;
    const uint16_t* bend = p.b + static_cast<int64_t>(p.E) * N * r;
    uint4 bmask[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) {
        const int n = r - 32 * k - 8 * g;     // ranks of this lane's eight that exist
        auto word = [&](int w) { return n >= 2 * w + 2 ? ~0u : (n == 2 * w + 1 ? 0xffffu : 0u); };
        bmask[k] = make_uint4(word(0), word(1), word(2), word(3));
    }
    const int tiles = (N + 127) / 128;
    const int per = (tiles + gridDim.y - 1) / gridDim.y;   // a multiple of W but for few tiles
    const int t1 = min(tiles, static_cast<int>(blockIdx.y + 1) * per);
    int ct = blockIdx.y * per + wave;
    // Small blocks keep one tile's operands ahead, the first of them from before U: with little else
    // in flight, a wave's time is the latency of its loads.
    constexpr int HB = RP == 64 && RB == 4 ? 1 : RB;   // row blocks whose base is held at a time (registers)
    constexpr bool AHEAD = RB == 2 && RP <= 32;
    uint4 bv[AHEAD ? 2 : 1][8][KS], base[AHEAD ? 2 : 1][HB][4];
    auto load_base = [&](int buf, int tile, int first) {   // rows 16 i + 4 g + x, columns 128 tile + 8 l16 ..
        const int n0 = tile * 128 + 8 * l16;
#pragma unroll
        for (int i = 0; i < HB; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                base[buf][i][x] = make_uint4(0, 0, 0, 0);
                if (p.base && first + i < nrb)
                    base[buf][i][x] = ld16_nt(p.base + static_cast<int64_t>(row0 + min(16 * (first + i) + 4 * g + x, rows - 1)) * N +
                                              (n0 < N ? n0 : 0));
            }
    };
    auto load_tile = [&](int buf, int tile) {
        load_base(buf, tile, 0);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int c = min(tile * 128 + 8 * l16 + t, N - 1);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int c0 = 32 * k + 8 * g;
                const uint16_t* src = be + static_cast<int64_t>(c) * r + c0;
                bv[buf][t][k] = make_uint4(0, 0, 0, 0);
                if (c0 < r) {
                    if (src + 8 <= bend) __builtin_memcpy(&bv[buf][t][k], src, 16);
                    else bv[buf][t][k] = gather8(src, 1, r - c0);
                }
            }
        }
    };
    if (AHEAD && ct < t1) load_tile(0, ct);

    // ---- U: fewer row blocks leave registers for more columns in flight
    {
        f32x4 acc[RB][NT];
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
        if (nrb == 1) adapter_u<NT, 1, NT == 1 ? 4 : (NT == 2 ? 2 : 1), W>(p, ae, row0, rows, wave, acc);
        else if (RB == 2 || nrb == 2) adapter_u<NT, 2, 1, W>(p, ae, row0, rows, wave, acc);
        else adapter_u<NT, RB, 1, W>(p, ae, row0, rows, wave, acc);
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (i < nrb) *reinterpret_cast<f32x4*>(&s_part[wave][16 * i + l16][16 * j + 4 * g]) = acc[i][j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * nrb * UW; i += W * 64) {
        const int row = i / UW, c = i % UW;
        float v = 0.0f;
        if (row < rows && c < r) {
#pragma unroll
            for (int w = 0; w < W; ++w) v += s_part[w][row][c];
        }
        const uint16_t h = f2bf(v);
        s_u[row][c] = h;
        if (row < rows && c < r && blockIdx.y == 0) p.u[static_cast<int64_t>(row0 + row) * r + c] = h;
    }
    __syncthreads();

    // ---- y
    bf16x8 uo[RB][KS];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int k = 0; k < KS; ++k)
            if (i < nrb) uo[i][k] = *reinterpret_cast<const bf16x8*>(&s_u[16 * i + l16][32 * k + 8 * g]);
    auto do_tile = [&](int buf, int tile) {
        const int n0 = tile * 128 + 8 * l16;
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint4& v = bv[buf][t][k];
                v = make_uint4(v.x & bmask[k].x, v.y & bmask[k].y, v.z & bmask[k].z, v.w & bmask[k].w);
            }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            if (i >= nrb) continue;
            if (HB < RB && i > 0) load_base(buf, tile, i);
            f32x4 d[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                d[t] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KS; ++k) d[t] = mfma16(uo[i][k], as_bf16x8(bv[buf][t][k]), d[t]);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int row = 16 * i + 4 * g + x;
                const uint4 bs = base[buf][i % HB][x];
                const uint32_t bw[4] = {bs.x, bs.y, bs.z, bs.w};
                uint32_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    o[q] = pack2(lo_f(bw[q]) + p.scale * d[2 * q][x], hi_f(bw[q]) + p.scale * d[2 * q + 1][x]);
                if (n0 < N && row < rows)
                    st16_nt(p.out + static_cast<int64_t>(row0 + row) * N + n0, make_uint4(o[0], o[1], o[2], o[3]));
            }
        }
    };
    if constexpr (AHEAD) {
        for (; ct < t1; ct += 2 * W) {
            if (ct + W < t1) load_tile(1, ct + W);
            do_tile(0, ct);
            if (ct + W >= t1) break;
            if (ct + 2 * W < t1) load_tile(0, ct + 2 * W);
            do_tile(1, ct + W);
        }
    } else {
        for (; ct < t1; ct += W) {
            load_tile(0, ct);
            do_tile(0, ct);
        }
    }
}

// ---------------------------------------------------------------- backward
//
// Four launches over 32-row blocks that start at each expert's first row:
//   1  output side: a unit is up to rows1 rows of one expert x a chunk of dy's
//      columns.  It reads dy once and makes both products of it: db (summed
//      over the rows in registers) and the chunk's part of du = scale dy b.
//   2  du: the chunks' parts added in order, rounded to bf16 for dx (bf16 itself:
//      relative error 0.00170 where a whole du would leave 0.00166; without a base 0.00234), and
//      kept whole as the sum of three bf16 values for da, whose output is fp32.
//   3  input side: a unit is up to rows2 rows of one expert x 512 columns of x:
//      da (summed in registers) and dx = base + du a.
//   4  experts with several units: their parts added in order; experts without
//      rows: zeros.
// A sum over rows needs the rows as the instruction's summed dimension: a lane
// loads the same 8 columns of 8 rows (256-byte row segments across 16 lanes)
// and pairs them up by byte permutes, so its 8 operands are 8 columns with 8
// rows each.
// Measured on 262144 rows, K 2048, N 4096, rank 64, and the memory traffic with it: 1 takes 0.62 ms
// (3.2 GB, 5.1 TB/s: dy, and 0.5 GB of du's parts), 2 takes 0.16 ms, 3 0.72 ms (4.0 GB, 5.6 TB/s: x, base, dx,
// and du once for each 512 columns), 4 0.04 ms.  At rank 16 (32768 rows, K 2048, N 1536) 29, 5, 86 and 9 us.
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

// The units of an expert's m rows: as many as m / unit_rows rounds to, of equal
// multiples of 32 rows.  Units of unit_rows with a short one after them make a few workgroups more than
// the CUs take at once, and all wait for those (32 experts of about 1024 rows, K 2048, N 1536, rank 16:
// 145 us so, 134 us here).
struct Units {
    int rows, n;
};
__device__ __forceinline__ Units units_of(int m, int unit_rows) {
    if (m < unit_rows + unit_rows / 2) return Units{(max(m, 1) - 1) / AD_BLK * AD_BLK + AD_BLK, m > 0 ? 1 : 0};
    const int n = m / unit_rows + (m % unit_rows >= unit_rows / 2 ? 1 : 0);
    const int rows = ((m - 1) / n / AD_BLK + 1) * AD_BLK;
    return Units{rows, (m - 1) / rows + 1};
}

// Unit i of the list of units of about unit_rows rows (e = -1 past its end).
__device__ __forceinline__ AdapterUnit find_unit(const AdapterParams& p, int unit_rows, int i) {
    const ExpertItem<3> it = find_item<3>(p.offsets, p.E, p.M, i, [&](int m) {
        const int units = units_of(m, unit_rows).n;
        return Counts<3>{{units, (m + AD_BLK - 1) / AD_BLK, units > 1 ? units : 0}};
    });
    const int part = i - it.before[0];
    const Units us = units_of(it.hi - it.lo, unit_rows);
    AdapterUnit u;
    u.e = it.e;
    u.row0 = it.lo + part * us.rows;
    u.rows = min(us.rows, it.hi - u.row0);
    u.blk0 = it.before[1] + part * (us.rows / AD_BLK);
    u.slot = us.n > 1 ? it.before[2] + part : -1;
    return u;
}

// 16 bytes at a wave-uniform base and a 32-bit byte offset of this lane.
__device__ __forceinline__ uint4 ld16_at(const uint16_t* base, uint32_t bytes) {
    return *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(base) + bytes);
}

__device__ __forceinline__ uint4 ld16_nt_at(const uint16_t* base, uint32_t bytes) {
    return ld16_nt(reinterpret_cast<const char*>(base) + bytes);
}

// Rows r0 .. r0 + R - 1 of the 32-row block at `block` (its first row, of row
// length ld), of which `left` rows exist (later ones repeat the last), columns
// c .. c + 7.  No branches: a load behind a branch would make the compiler
// wait for every load before the next use of any.
template <int R>
__device__ __forceinline__ void load_rows(const uint16_t* block, int ld, int r0, int left, int c, uint4 (&v)[R]) {
#pragma unroll
    for (int t = 0; t < R; ++t) v[t] = ld16_nt_at(block, static_cast<uint32_t>(min(r0 + t, left - 1) * ld + c) * 2);
}
// Rows past `left`, and columns that do not exist, are zero.
template <int R>
__device__ __forceinline__ void mask_rows(int r0, int left, bool in, uint4 (&v)[R]) {
#pragma unroll
    for (int t = 0; t < R; ++t) v[t] = and4(v[t], in && r0 + t < left ? ~0u : 0u);
}

// A wave's registers for the token rows are refilled for the next block as
// soon as they are consumed, so that 8 KiB a wave are on their way for most of
// the time.
template <int RP>
__global__ __launch_bounds__(ad_groups(RP) * ad_split(RP) * 64) void adapter_dy_kernel(const AdapterParams p) {
    constexpr int RS = ad_split(RP), NG = ad_groups(RP);
    constexpr int NT = RP / 16 / RS;             // rank tiles of a wave
    constexpr int MIN_THREADS = ad_groups_min(RP) * RS * 64;
    // each column group's 32 x 128 tile of dy; 16-byte chunk c of row i at c ^ (i & 15).  Two for groups of
    // two waves, which each bring half of the next block's rows while they compute.
    __shared__ __attribute__((aligned(16))) uint16_t s_dy[RS][NG][AD_BLK * AD_WCOLS];
    __shared__ __attribute__((aligned(16))) uint16_t s_u[2][AD_BLK * RP];                      // U of a block
    __shared__ __attribute__((aligned(16))) float s_du[2][NG][AD_BLK][RP + 4];   // the groups' parts of du
    const int chunk = blockIdx.x % p.chunks1;   // neighbouring workgroups share rows
    const AdapterUnit un = find_unit(p, p.rows1, blockIdx.x / p.chunks1);
    if (un.e < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int nthreads = blockDim.x, ng = nthreads / (64 * RS);
    const int grp = wave / RS, r0 = wave % RS * (RP / RS);   // the wave's columns and first rank
    const int l16 = lane & 15, g = lane >> 4;
    const int N = p.N, r = p.r;
    const int c0 = (chunk * ng + grp) * AD_WCOLS;
    const bool in = c0 + 8 * l16 < N;
    const int cl = in ? c0 + 8 * l16 : 0;         // the lane's columns
    const bool whole = c0 + AD_WCOLS <= N;
    const uint16_t* be = p.b + static_cast<int64_t>(un.e) * N * r;
    const uint16_t* dy0 = p.dy + static_cast<int64_t>(un.row0) * N;
    const uint16_t* ue = p.u + static_cast<int64_t>(un.row0) * r;

    // U of a block is 32 r values in a row: 16 bytes a thread, from any 2-byte boundary.  A load that would
    // reach past the tensor's end takes its values one by one.
    constexpr int UPT = (AD_BLK * RP / 8 + MIN_THREADS - 1) / MIN_THREADS;
    const uint16_t* uend = p.u + static_cast<int64_t>(p.M) * r;
    uint4 uv[UPT];
    auto load_u = [&](int row) {
        const uint16_t* from = ue + static_cast<int64_t>(row) * r;
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const int el = (tid + i * nthreads) * 8;
            if (el >= AD_BLK * r) continue;
            const int64_t have = uend - (from + el);
            if (have >= 8) __builtin_memcpy(&uv[i], from + el, 16);
            else uv[i] = gather8(have > 0 ? from + el : ue, 1, static_cast<int>(have));
        }
    };
    auto put_u = [&](int buf) {
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const int el = (tid + i * nthreads) * 8;
            if (el < AD_BLK * r) *reinterpret_cast<uint4*>(&s_u[buf][el]) = uv[i];
        }
    };
    // U as the operand of db: rank 16 j + l16 (a rank past r gives columns that are not kept), rows 8 g ..
    auto read_u = [&](int buf, int j, int left) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = s_u[buf][(8 * g + i) * r + r0 + 16 * j + l16];
            if (left < AD_BLK && 8 * g + i >= left) w[i] = 0;     // rows past the end: not U's
        }
        return as_bf16x8(make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16)));
    };
    constexpr int TR = 8 / RS;                   // of each 32-row block a lane loads rows rl .. rl + TR - 1
    const int rl = 8 * g + wave % RS * TR;
    uint4 t[TR];
    auto load_t = [&](int row) { load_rows<TR>(dy0 + static_cast<int64_t>(row) * N, N, rl, un.rows - row, cl, t); };
    auto put_t = [&](int row, int buf) {
        if (!whole || row + AD_BLK > un.rows) mask_rows<TR>(rl, un.rows - row, in, t);
#pragma unroll
        for (int i = 0; i < TR; ++i)
            *reinterpret_cast<uint4*>(&s_dy[buf % RS][grp][(rl + i) * AD_WCOLS + ((l16 ^ ((rl + i) & 15)) << 3)]) = t[i];
    };
    load_u(0);
    load_t(0);
    bf16x8 bw[4][NT];   // b as the operand of du: rank 16 j + l16, columns c0 + 32 k + 8 g ..
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int c = c0 + 32 * k + 8 * g, rr = r0 + 16 * j + l16;
            bw[k][j] = as_bf16x8(gather8(be + static_cast<int64_t>(min(c, N - 1)) * r + min(rr, r - 1), r, rr < r ? N - c : 0));
        }
        if (NT * (k + 1) % 4 == 0) __builtin_amdgcn_sched_barrier(0);   // 32 loads at a time
    }
    f32x4 acc[8][NT];
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[c][j] = f32x4{0, 0, 0, 0};
    put_u(0);
    const int last = (un.rows - 1) / AD_BLK * AD_BLK;
    if constexpr (RS > 1) {
        put_t(0, 0);
        load_u(min(AD_BLK, last));
        load_t(min(AD_BLK, last));
    }
    __syncthreads();

    // the waves' parts of du of the block at `row`, added up and stored
    auto store_du = [&](int row, int buf) {
        float* part = p.du_part + ((static_cast<int64_t>(chunk) * p.blocks + un.blk0 + row / AD_BLK) * AD_BLK) * RP;
        for (int i = tid; i < AD_BLK * RP / 4; i += nthreads) {
            const int rr = i / (RP / 4), c = i % (RP / 4) * 4;
            f32x4 sum = *reinterpret_cast<const f32x4*>(&s_du[buf][0][rr][c]);
            for (int w = 1; w < ng; ++w) sum += *reinterpret_cast<const f32x4*>(&s_du[buf][w][rr][c]);
            *reinterpret_cast<f32x4*>(part + rr * RP + c) = sum;
        }
    };
    int buf = 0;
    for (int row = 0; row < un.rows; row += AD_BLK, buf ^= 1) {
        const int ahead = min(row + AD_BLK, last);
        uint4 tr[8];
        const uint16_t* tile = s_dy[buf % RS][grp];
        if constexpr (RS == 1) {
            put_t(row, buf);
            transpose8(t, tr);
        } else {
            uint4 rows8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                rows8[i] = *reinterpret_cast<const uint4*>(tile + (8 * g + i) * AD_WCOLS + ((l16 ^ ((8 * g + i) & 15)) << 3));
            transpose8(rows8, tr);
        }
        // Memory operations complete in order: the stores go out before the next loads, whose
        // wait (in the next block) would otherwise be for the stores too.
        if (row > 0) store_du(row - AD_BLK, buf ^ 1);
        if constexpr (RS == 1) {
            load_u(ahead);
            __builtin_amdgcn_sched_barrier(0);   // t is free: nothing of the refill moves above
            load_t(ahead);
            __builtin_amdgcn_sched_barrier(0);   // nor does it wait for what follows
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const bf16x8 ut = read_u(buf, j, un.rows - row);
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
                *reinterpret_cast<f32x4*>(&s_du[buf][grp][16 * h + l16][r0 + 16 * j + 4 * g]) = du[h][j];
        put_u(buf ^ 1);
        if constexpr (RS > 1) {
            // the next block's rows into the other tile, and the loads of the one after it
            put_t(ahead, buf ^ 1);
            const int after = min(row + 2 * AD_BLK, last);
            load_u(after);
            load_t(after);
        }
        // The waves' parts are in; the next block's go to the other buffers.  Only LDS is
        // handed over here, so the rows on their way are not waited for.
        block_barrier();
    }
    store_du(last, buf ^ 1);
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
                const int n = c0 + 8 * (4 * g + x) + c, rr = r0 + 16 * j + l16;
                if (n < N && rr < r) {
                    float* o = out + static_cast<int64_t>(n) * r + rr;
                    const float v = p.scale * acc[c][j][x];
                    *o = add ? *o + v : v;
                }
            }
}

// du of every block from its parts, in chunk order; rows past an expert's end
// are zero already.  A workgroup takes 1024 or more values at a time, read as
// they lie (rank fastest) and written so and transposed.
template <int RP>
__global__ __launch_bounds__(256) void adapter_du_kernel(const AdapterParams p) {
    constexpr int UW = RP < 32 ? 32 : RP;
    constexpr int VALS = AD_BLK * RP;                     // values of a block
    constexpr int NB = VALS < 1024 ? 1024 / VALS : 1;     // blocks at a time
    __shared__ int s_off[GG_KMAX_EXPERTS + 1];
    __shared__ int s_blk[GG_KMAX_EXPERTS + 1];
    __shared__ __attribute__((aligned(16))) uint16_t s_t[3][NB * RP][AD_BLK + 8];
    prefix_experts(p.offsets, p.E, p.M, s_off, s_blk, [](int m) { return (m + AD_BLK - 1) / AD_BLK; });
    const int total = uni(s_blk[p.E]);
    for (int blk = blockIdx.x * NB; blk < total; blk += gridDim.x * NB) {
#pragma unroll
        for (int i = 0; i < NB * VALS / 1024; ++i) {
            const int v4 = (i * 256 + threadIdx.x) * 4, nb = v4 / VALS, row = v4 % VALS / RP, c = v4 % RP;
            if (blk + nb >= total) continue;
            const float* src = p.du_part + static_cast<int64_t>(blk) * VALS + v4;
            f32x4 v = {0, 0, 0, 0};
            for (int k = 0; k < p.chunks1; ++k)
                v += *reinterpret_cast<const f32x4*>(src + static_cast<int64_t>(k) * p.blocks * VALS);
            uint32_t hi[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                // ranks that do not exist are zero: the padded operands give them NaN where dy is infinite
                const float d = c + x < p.r ? v[x] * p.scale : 0.0f;
                hi[x] = f2bf(d);
                // an infinity is its first part alone: infinity - infinity is NaN
                const float rest = __builtin_isinf(bf2f(hi[x])) ? 0.0f : d - bf2f(hi[x]);
                const uint16_t mid = f2bf(rest);
                s_t[0][nb * RP + c + x][row] = static_cast<uint16_t>(hi[x]);
                s_t[1][nb * RP + c + x][row] = mid;
                s_t[2][nb * RP + c + x][row] = f2bf(rest - bf2f(mid));
            }
            uint16_t* d = p.du + ((static_cast<int64_t>(blk) + nb) * AD_BLK + row) * UW + c;
            *reinterpret_cast<uint2*>(d) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
            if (RP < UW) *reinterpret_cast<uint2*>(d + RP) = make_uint2(0, 0);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < NB * 3 * RP * AD_BLK / 8; i += 256) {
            const int nb = i / (3 * RP * AD_BLK / 8), w = i % (3 * RP * AD_BLK / 8);
            const int q = w / (RP * AD_BLK / 8), c = w / (AD_BLK / 8) % RP, row = w % (AD_BLK / 8) * 8;
            if (blk + nb < total)
                *reinterpret_cast<uint4*>(p.du_t + (((static_cast<int64_t>(blk) + nb) * 3 + q) * RP + c) * AD_BLK + row) =
                    *reinterpret_cast<const uint4*>(&s_t[q][nb * RP + c][row]);
        }
        __syncthreads();
    }
}

template <int RP>
__global__ __launch_bounds__(256) void adapter_dx_kernel(const AdapterParams p) {
    constexpr int NT = RP / 16;
    constexpr int UW = RP < 32 ? 32 : RP;
    constexpr int KS = UW / 32;
    // a as the operand of dx, for each wave: columns c0 + 8 l16 + t, ranks 32 k + 8 g ..
    __shared__ __attribute__((aligned(16))) uint4 s_aw[4][8][KS][64];
    const int chunk = blockIdx.x % p.chunks2;
    const AdapterUnit un = find_unit(p, p.rows2, blockIdx.x / p.chunks2);
    if (un.e < 0) return;
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int K = p.K, r = p.r;
    const int c0 = (chunk * 4 + wave) * AD_WCOLS;
    if (c0 >= K) return;                        // no barrier below: each wave keeps to its own part of LDS
    const bool in = c0 + 8 * l16 < K, whole = c0 + AD_WCOLS <= K;
    const int cl = in ? c0 + 8 * l16 : 0;
    const uint16_t* ae = p.a + static_cast<int64_t>(un.e) * r * K;

    uint4 x[8], base[2][4];
    bf16x8 dt[3][NT], dr[2][KS];
    const uint16_t* x0 = p.x + static_cast<int64_t>(un.row0) * K;
    // without a base its place is taken by x, cleared: the loads stay the same
    const uint16_t* base0 = (p.base ? p.base : p.x) + static_cast<int64_t>(un.row0) * K;
    const uint32_t keep = p.base ? ~0u : 0u;
    auto load_base = [&](int row) {   // rows 16 i + 4 g + x of the block at `row`
        const uint16_t* from = base0 + static_cast<int64_t>(row) * K;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                base[i][x] = ld16_nt_at(from, static_cast<uint32_t>(min(16 * i + 4 * g + x, un.rows - row - 1) * K + cl) * 2);
    };
    auto load_dt = [&](int row) {
        const uint16_t* from = p.du_t + (static_cast<int64_t>(un.blk0) + row / AD_BLK) * 3 * RP * AD_BLK;
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                dt[q][j] = as_bf16x8(ld16_at(from, ((q * RP + 16 * j + l16) * AD_BLK + 8 * g) * 2));
    };
    auto load_dr = [&](int row) {
        const uint16_t* from = p.du + (static_cast<int64_t>(un.blk0) + row / AD_BLK) * AD_BLK * UW;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < KS; ++k) dr[i][k] = as_bf16x8(ld16_at(from, ((16 * i + l16) * UW + 32 * k + 8 * g) * 2));
    };
    load_rows<8>(x0, K, 8 * g, un.rows, cl, x);
    load_dt(0);
    load_base(0);
    load_dr(0);
#pragma unroll 4
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int rr = 32 * k + 8 * g;
            s_aw[wave][t][k][lane] = gather8(ae + static_cast<int64_t>(min(rr, r - 1)) * K + cl + t, K, in ? r - rr : 0);
        }
    f32x4 acc[8][NT];
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[c][j] = f32x4{0, 0, 0, 0};

    const int last = (un.rows - 1) / AD_BLK * AD_BLK;
    for (int row = 0; row < un.rows; row += AD_BLK) {
        const int ahead = min(row + AD_BLK, last);
        if (!whole || row + AD_BLK > un.rows) mask_rows<8>(8 * g, un.rows - row, in, x);
        uint4 tr[8];
        transpose8(x, tr);
        __builtin_amdgcn_sched_barrier(0);   // x is free: nothing of the refill moves above
        load_rows<8>(x0 + static_cast<int64_t>(ahead) * K, K, 8 * g, un.rows - ahead, cl, x);
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int q = 2; q >= 0; --q) acc[c][j] = mfma16(as_bf16x8(tr[c]), dt[q][j], acc[c][j]);
        __builtin_amdgcn_sched_barrier(0);
        load_dt(ahead);
        int at = lane;
        asm volatile("" : "+v"(at));         // a's operands are read anew in every block, not held
        f32x4 d[2][8];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) d[i][t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const bf16x8 aw = as_bf16x8(s_aw[wave][t][k][at]);
#pragma unroll
                for (int i = 0; i < 2; ++i) d[i][t] = mfma16(dr[i][k], aw, d[i][t]);
            }
        uint16_t* to = p.out + static_cast<int64_t>(un.row0 + row) * K;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint4 bs = and4(base[i][x], keep);
                const uint32_t bw[4] = {bs.x, bs.y, bs.z, bs.w};
                uint32_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    o[q] = pack2(lo_f(bw[q]) + d[i][2 * q][x], hi_f(bw[q]) + d[i][2 * q + 1][x]);
                const int rr = 16 * i + 4 * g + x;
                if (in && row + rr < un.rows)
                    st16_nt(to + static_cast<uint32_t>(rr * K + cl), make_uint4(o[0], o[1], o[2], o[3]));
            }
        __builtin_amdgcn_sched_barrier(0);
        load_dr(ahead);
        load_base(ahead);
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
    if (m > 0 ? units_of(m, unit_rows).n == 1 : p.accumulate) return;   // written by its one unit, or nothing to add
    int s0 = 0, n = 0;
    if (m > 0) {
        prefix_experts(p.offsets, p.E, p.M, s_off, s_slot,
                       [&](int m) {
                           const int units = units_of(m, unit_rows).n;
                           return units > 1 ? units : 0;
                       });
        s0 = uni(s_slot[e]);
        n = uni(s_slot[e + 1]) - s0;
    }
    const int64_t size = static_cast<int64_t>(p.r) * (blockIdx.y ? p.K : p.N);   // a multiple of 4
    const float* part = blockIdx.y ? p.da_part : p.db_part;
    float* out = (blockIdx.y ? p.da : p.db) + e * size;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < size;
         i += static_cast<int64_t>(gridDim.x) * 1024) {
        f32x4 v = {0, 0, 0, 0};
        const float* at = part + s0 * size + i;
        int k = 0;
        for (; k + 4 <= n; k += 4) {
            f32x4 w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = *reinterpret_cast<const f32x4*>(at + (k + q) * size);
#pragma unroll
            for (int q = 0; q < 4; ++q) v += w[q];
        }
        for (; k < n; ++k) v += *reinterpret_cast<const f32x4*>(at + k * size);
        f32x4* o = reinterpret_cast<f32x4*>(out + i);
        if (p.accumulate) v += *o;
        *o = v;
    }
}

// ---------------------------------------------------------------- launchers
template <int RP, int RB>
static hipError_t forward_rows(const AdapterParams& p, int num_cu, hipStream_t s) {
    constexpr int W = af_waves(RB);
    const int64_t blocks = static_cast<int64_t>(p.M) / (16 * RB) + (p.M < p.E ? p.M : p.E);
    // sixteen waves for each CU where the rows alone give fewer, down to one tile a wave
    const int64_t tiles = (p.N + 127) / 128;
    int64_t split = 16 / W * static_cast<int64_t>(num_cu) / blocks;
    split = split < 1 ? 1 : split;
    const int64_t per = ((tiles + split - 1) / split + W - 1) / W * W;
    hipLaunchKernelGGL((adapter_forward_kernel<RP, RB>),
                       dim3(static_cast<unsigned>(blocks), static_cast<unsigned>((tiles + per - 1) / per)), dim3(W * 64), 0, s,
                       p);
    return hipGetLastError();
}

// Small blocks where the experts have at most 128 rows each on average (128 experts, K = N = 2048, rank 32:
// of 100 rows 46 us, 59 us with large blocks; of 200 rows 91 us, and 76 us).
template <int RP>
static hipError_t forward_of(const AdapterParams& p, int num_cu, hipStream_t s) {
    return p.M <= 128 * static_cast<int64_t>(p.E) ? forward_rows<RP, 2>(p, num_cu, s) : forward_rows<RP, 4>(p, num_cu, s);
}

hipError_t launch_adapter_forward(const AdapterParams& p, int num_cu, hipStream_t s) {
    switch (ad_rank_p(p.r)) {
        case 16: return forward_of<16>(p, num_cu, s);
        case 32: return forward_of<32>(p, num_cu, s);
        default: return forward_of<64>(p, num_cu, s);
    }
}

template <int RP>
static hipError_t backward_of(AdapterParams p, int num_cu, hipStream_t s) {
    const int64_t few = p.M < p.E ? p.M : p.E;
    p.chunks1 = ad_chunks(p.N, RP);
    p.chunks2 = (p.K + 4 * AD_WCOLS - 1) / (4 * AD_WCOLS);
    // the columns of dy spread evenly over its chunks
    const int parts = (p.N + AD_WCOLS - 1) / AD_WCOLS, even = (parts + p.chunks1 - 1) / p.chunks1;
    const int groups = even > ad_groups_min(RP) ? even : ad_groups_min(RP);
    hipError_t st;
    if (p.M > 0) {
        hipLaunchKernelGGL((adapter_dy_kernel<RP>), dim3(static_cast<unsigned>((p.M / p.rows1 + few) * p.chunks1)),
                           dim3(static_cast<unsigned>(groups * ad_split(RP)) * 64), 0, s, p);
        if ((st = hipGetLastError()) != hipSuccess) return st;
        const int64_t most = static_cast<int64_t>(num_cu) * 6;
        hipLaunchKernelGGL((adapter_du_kernel<RP>), dim3(static_cast<unsigned>(p.blocks < most ? p.blocks : most)), dim3(256),
                           0, s, p);
        if ((st = hipGetLastError()) != hipSuccess) return st;
        hipLaunchKernelGGL((adapter_dx_kernel<RP>), dim3(static_cast<unsigned>((p.M / p.rows2 + few) * p.chunks2)),
                           dim3(256), 0, s, p);
        if ((st = hipGetLastError()) != hipSuccess) return st;
    }
    const int64_t width = p.N > p.K ? p.N : p.K, gx = (width * p.r / 4 + 511) / 512;
    hipLaunchKernelGGL(adapter_join_kernel, dim3(static_cast<unsigned>(gx < 64 ? gx : 64), 2, static_cast<unsigned>(p.E)),
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
