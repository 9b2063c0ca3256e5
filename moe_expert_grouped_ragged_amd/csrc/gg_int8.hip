// 8-bit expert products on CDNA4: token quantization (with the activation or
// its derivative fused in), the packed weight layout, and the ragged grouped
// int8 product.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gg_device.h"
#include "gg_int8.h"
#include "gg_kernels.h"

namespace gg {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(16))) int i32x16;
typedef __attribute__((ext_vector_type(4))) float f32x4;

// ---------------------------------------------------------------- quantization
//
// Per row: top = max|v|, s = top / 127, q = rint(127 v / top) to nearest even;
// a zero row gives s = 0, q = 0, and a row with a NaN or infinity s = NaN,
// q = 0, so that its products are NaN and no other row's are.  The quotient (a
// product with 1/top and one residual correction) rounds as the exact one does:
// with v = a 2^i and top = b 2^j, 8 bits each, 127 v is exact, and where
// 127 v / top is not a tie k + 1/2 it differs from one by
// |254 a - (2k + 1) b 2^d| / (2 b 2^d) >= 1 / (2 b 2^d) (d = j - i), which is the
// quotient divided by 254 a, above 2^-16 of it; the corrected quotient is within 2^-23.
// Rows whose top is far from one are scaled by a power of two first, so 1/top
// neither overflows nor loses bits.
//
// A wavefront takes a row at a time; its bf16 values stay in registers between
// the maximum and the rounding (rows of more than NC * 64 units are computed
// twice).  For large batches of the light modes it takes two neighbouring
// rows: pairs of lanes then exchange halves, so that a store is 16 bytes a
// lane and whole 128-byte lines of the two rows in the product's layout (262144 x
// 4096, 3.2 GB: 560 us, 760 us a row at a time; with a derivative or column
// scales in front, and in small batches, the second row costs more than it gives: 32768 x
// 1536 with the derivative 65 us, 105 us in pairs).
template <int MODE>
struct QuantUnit {
    static constexpr int HALVES = MODE == Q_DGLU ? 2 : 1;   // groups of 8 values a lane makes at a time
};

// The bf16 values of unit c of row r (groups of 8: x, A, or dH1's gate and up parts), and their copy to v_out.
template <int MODE>
__device__ __forceinline__ void quant_unit(const QuantParams& p, int64_t r, int c, bool store,
                                           uint4 (&w)[QuantUnit<MODE>::HALVES]) {
    if constexpr (MODE == Q_PLAIN || MODE == Q_SCALED) {
        w[0] = ld16_nt(p.x + r * p.K + c * 8);
    } else if constexpr (MODE == Q_GLU) {
        const uint16_t* row = p.x + r * 2 * p.K + c * 8;
        const uint4 g4 = ld16_nt(row), u4 = ld16_nt(row + p.K);
        const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
        uint32_t aw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {   // the arithmetic of the FC1 epilogue
                const float g = y ? hi_f(gw[i]) : lo_f(gw[i]);
                const float u = y ? hi_f(uw[i]) : lo_f(uw[i]);
                const float sg = g * __builtin_amdgcn_rcpf(1.0f + __expf(-(p.slope * g)));
                a[y] = sg * u;
            }
            aw[i] = pack2(a[0], a[1]);
        }
        w[0] = make_uint4(aw[0], aw[1], aw[2], aw[3]);
        if (store) *reinterpret_cast<uint4*>(p.v_out + r * p.K + c * 8) = w[0];
    } else {
        const int F = p.K / 2;
        const uint16_t* hrow = p.h1 + r * p.K + c * 8;
        const uint4 g4 = ld16_nt(hrow), u4 = ld16_nt(hrow + F), d4 = ld16_nt(p.x + r * F + c * 8);
        const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
        const uint32_t dw[4] = {d4.x, d4.y, d4.z, d4.w};
        uint32_t og[4], ou[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float dg[2], du[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {   // the arithmetic of the dgrad FC2 epilogue
                const float g = y ? hi_f(gw[i]) : lo_f(gw[i]);
                const float u = y ? hi_f(uw[i]) : lo_f(uw[i]);
                const float da = y ? hi_f(dw[i]) : lo_f(dw[i]);
                const float sgm = __builtin_amdgcn_rcpf(1.0f + __expf(-(p.slope * g)));
                dg[y] = da * u * sgm * (1.0f + p.slope * g * (1.0f - sgm));
                du[y] = da * g * sgm;
            }
            og[i] = pack2(dg[0], dg[1]);
            ou[i] = pack2(du[0], du[1]);
        }
        w[0] = make_uint4(og[0], og[1], og[2], og[3]);
        w[1] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
        if (store) {
            uint16_t* o = p.v_out + r * p.K + c * 8;
            *reinterpret_cast<uint4*>(o) = w[0];
            *reinterpret_cast<uint4*>(o + F) = w[1];
        }
    }
}

// Eight bf16 values as floats, times their column scales (cs null: no scales).
__device__ __forceinline__ void quant_vals(uint4 w, const float* cs, float (&v)[8]) {
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = lo_f(ww[i]);
        v[2 * i + 1] = hi_f(ww[i]);
    }
    if (cs) {
        const float4 c0 = *reinterpret_cast<const float4*>(cs), c1 = *reinterpret_cast<const float4*>(cs + 4);
        const float cf[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= cf[i];
    }
}

// Eight values to eight int8: t = v * c127 (127 times the row's power of two),
// the corrected quotient t / top, then the sum with 1.5 * 2^23, whose rounding
// is to the nearest even integer and whose low byte is that integer.
struct QuantScale {
    float c127, top, inv;
    bool zero;   // a row of zeros, or one that is not finite
};
__device__ __forceinline__ uint2 quant8(const float (&v)[8], const QuantScale& s) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = v[i] * s.c127;
        const float q0 = t * s.inv;
        const float q = __builtin_fmaf(__builtin_fmaf(-q0, s.top, t), s.inv, q0);
        b[i] = __builtin_bit_cast(uint32_t, q + 12582912.0f);
    }
    auto four = [](uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {   // the low bytes
        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(x3, x2, 0x0c0c0400u), __builtin_amdgcn_perm(x1, x0, 0x0c0c0400u),
                                     0x05040100u);
    };
    if (s.zero) return make_uint2(0, 0);
    return make_uint2(four(b[0], b[1], b[2], b[3]), four(b[4], b[5], b[6], b[7]));
}

// top: the largest |v| of the row as bits (a NaN is larger than infinity, which is larger than any number).
__device__ __forceinline__ QuantScale quant_scale(uint32_t bits) {
    QuantScale s;
    const float top = __builtin_bit_cast(float, bits);
    // a power of two that brings the row near one where it is far from it
    const float pw = top < 0x1p-90f ? 0x1p64f : (top > 0x1p90f ? 0x1p-64f : 1.0f);
    s.c127 = 127.0f * pw;
    s.top = top * pw;
    s.inv = 1.0f / s.top;
    s.zero = bits == 0 || bits >= 0x7f800000u;
    return s;
}

template <int MODE, int NC, int Y>   // NC = 0: any width, values computed twice; Y: rows a wave takes at a time
__global__ __launch_bounds__(256) void quant_rows_kernel(const QuantParams p) {
    __shared__ int s_off[GG_KMAX_EXPERTS + 1];
    constexpr int HALVES = QuantUnit<MODE>::HALVES;
    constexpr bool SCALES = MODE == Q_SCALED || MODE == Q_DGLU;
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = p.M;
    if (p.offsets) {
        for (int e = threadIdx.x; e <= p.E; e += 256) {
            int64_t o = p.offsets[e];
            o = o < 0 ? 0 : (o > p.M ? p.M : o);
            s_off[e] = static_cast<int>(o);
        }
        __syncthreads();
        lo = s_off[0];
        hi = s_off[p.E];
    }
    const int units = p.K / (8 * HALVES), half = p.K / 2;
    for (int64_t r0 = i8_first_row<Y>(lo, hi) + Y * (static_cast<int64_t>(blockIdx.x) * 4 + uni(threadIdx.x >> 6)); r0 < hi;
         r0 += static_cast<int64_t>(gridDim.x) * 4 * Y) {
        int64_t row[Y];
        i8_rows_at<Y>(r0, lo, hi, row);
        const bool keep = p.v_out != nullptr;
        const float* cs[Y] = {};
        if constexpr (SCALES) {
#pragma unroll
            for (int y = 0; y < Y; ++y)
                cs[y] = p.cs + static_cast<int64_t>(uni(find_expert_wave(s_off, p.E, static_cast<int>(row[y])))) * p.cs_ld;
        }
        uint4 w[Y][NC ? NC : 1][HALVES];
        float f[SCALES ? Y : 1][SCALES && NC ? NC : 1][HALVES][8];   // scaled values, made once
        uint32_t m[Y] = {};
        auto top_of = [&](int y, int j, int c) {
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                float v[8];
                quant_vals(w[y][j][h], SCALES ? cs[y] + h * half + c * 8 : nullptr, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    m[y] = max(m[y], __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);
                    if constexpr (SCALES) f[y][j][h][i] = v[i];
                }
            }
        };
        if constexpr (NC > 0) {
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int y = 0; y < Y; ++y) {   // repeated last units do not change the maximum
                    const int c = lane + 64 * j;
                    quant_unit<MODE>(p, row[y], min(c, units - 1), keep && c < units, w[y][j]);
                }
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int y = 0; y < Y; ++y) top_of(y, j, min(lane + 64 * j, units - 1));
        } else {
            for (int c = lane; c < units; c += 64)
#pragma unroll
                for (int y = 0; y < Y; ++y) {
                    quant_unit<MODE>(p, row[y], c, keep, w[y][0]);
                    top_of(y, 0, c);
                }
        }
        QuantScale sc[Y];
#pragma unroll
        for (int y = 0; y < Y; ++y) {
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1)
                m[y] = max(m[y], static_cast<uint32_t>(__shfl_xor(static_cast<int>(m[y]), d, 64)));
            sc[y] = quant_scale(m[y]);
            if (lane == 0) p.s[row[y]] = m[y] < 0x7f800000u ? __builtin_bit_cast(float, m[y]) / 127.0f : __builtin_nanf("");
        }
        if constexpr (Y == 2 && NC > 0) {
            // The floats are made again from the kept bf16 values: held over the reductions they would take twice the
            // registers.
#pragma unroll
            for (int y = 0; y < Y; ++y)
#pragma unroll
                for (int j = 0; j < NC; ++j)
#pragma unroll
                    for (int h = 0; h < HALVES; ++h)
                        asm volatile("" : "+v"(w[y][j][h].x), "+v"(w[y][j][h].y), "+v"(w[y][j][h].z), "+v"(w[y][j][h].w));
        }
        auto at = [&](int64_t r, int c) { return p.q + r * p.q_row + (c >> 6) * p.q_block + (c & 63); };
        // unit c of the rows; lanes past the end take part in the exchange of a pair with zeros
        auto put = [&](int c, int j) {
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                uint2 q[Y];
#pragma unroll
                for (int y = 0; y < Y; ++y) {
                    if constexpr (SCALES) {
                        q[y] = quant8(f[y][j][h], sc[y]);
                    } else {
                        float v[8];
                        quant_vals(w[y][j][h], nullptr, v);
                        q[y] = quant8(v, sc[y]);
                    }
                    if (c >= units) q[y] = make_uint2(0, 0);
                }
                const int col = h * half + c * 8;
                if constexpr (Y == 2) {
                    // even lanes: 16 bytes of the first row; odd lanes: of the second
                    const bool odd = lane & 1;
                    const uint2 send = odd ? q[0] : q[1];
                    const uint2 got = make_uint2(__builtin_amdgcn_mov_dpp(send.x, 0xb1, 0xf, 0xf, true),     // the other
                                                 __builtin_amdgcn_mov_dpp(send.y, 0xb1, 0xf, 0xf, true));    // lane of the pair
                    const uint4 o = odd ? make_uint4(got.x, got.y, q[1].x, q[1].y) : make_uint4(q[0].x, q[0].y, got.x, got.y);
                    if ((c & ~1) < units) *reinterpret_cast<uint4*>(at(row[odd], col & ~15)) = o;
                } else if (c < units) {
                    *reinterpret_cast<uint2*>(at(row[0], col)) = q[0];
                }
            }
        };
        if constexpr (NC > 0) {
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                put(lane + 64 * j, j);
            }
        } else {
            for (int c = lane; c - lane < units; c += 64) {
#pragma unroll
                for (int y = 0; y < Y; ++y) {
                    quant_unit<MODE>(p, row[y], min(c, units - 1), false, w[y][0]);
                    if constexpr (SCALES) top_of(y, 0, min(c, units - 1));
                }
                put(c, 0);
            }
        }
        const int pad = (p.width - p.K) / 8;   // below 16
        if (lane < Y * pad)
            *reinterpret_cast<uint2*>(at(row[lane % Y], p.K + lane / Y * 8)) = make_uint2(0, 0);
    }
}

// ---------------------------------------------------------------- packing
__global__ void int8_pack_kernel(const int8_t* __restrict__ q, const float* __restrict__ s, int E, int N, int K,
                                 int transposed, int8_t* __restrict__ packed, float* __restrict__ scales, int ns) {
    const int rows = transposed ? K : N, cont = transposed ? N : K;
    const int64_t nb = (rows + I8_ROWS - 1) / I8_ROWS, ks = (cont + I8_PAD - 1) / I8_PAD * (I8_PAD / I8_STEP);
    const int64_t total = static_cast<int64_t>(E) * nb * ks * 64;   // 16-byte operands
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    for (int64_t i = first; i < total; i += step) {
        const int l = static_cast<int>(i & 63);
        const int64_t blk = i >> 6;
        const int st = static_cast<int>(blk % ks);
        const int b = static_cast<int>(blk / ks % nb);
        const int64_t e = blk / ks / nb;
        const int row = b * I8_ROWS + (l & 31), c0 = st * I8_STEP + 16 * (l >> 5);
        const int8_t* m = q + e * N * K;
        uint32_t w[4] = {0, 0, 0, 0};
        if (row < rows) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int c = c0 + j;
                if (c < cont) {
                    const int8_t x = transposed ? m[static_cast<int64_t>(c) * K + row] : m[static_cast<int64_t>(row) * K + c];
                    w[j >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(x)) << (8 * (j & 3));
                }
            }
        }
        *reinterpret_cast<uint4*>(packed + i * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    for (int64_t i = first; i < static_cast<int64_t>(E) * ns; i += step) {
        const int64_t e = i / ns;
        const int n = static_cast<int>(i - e * ns);
        scales[i] = n < N ? s[e * N + n] : 0.0f;
    }
}

// ---------------------------------------------------------------- product
//
// The sums are exact in 32-bit integers, so the kernels below give the same
// bits.  The rows of a large expert run as tiles (the last may be partial);
// a remainder of few rows (all rows of a small expert) runs as streaming
// items.
//
// Streaming items: a group of rows of one expert x a range of output columns,
// for which each weight byte is read once.  A group holds up to 96 rows, or in
// the tiles' launch what LDS holds of the summed width where that is less (64 rows up to
// 2048 columns, 32 up to 4096): an expert of more rows reads its weights for each group.
// A wave takes 32 columns at a time over the whole summed dimension, its weights
// one coalesced 1 KiB load a step.  Bound by the weights' bytes.

// Rows of an expert that tiles of `tile` rows cover (0: there are no tiles).  256-row tiles leave a remainder
// of at most 96 rows (32768 rows over 32 experts, K 1536, N 2048: 164 us, 173 us with at most 32); 128-row tiles,
// which run where there is little work, take all of an expert of more than 64 rows, or nothing (128 experts of
// 80 rows, K 2048, N 1536: 124 us, 178 us with more than 96; of 24 rows 87 us, 94 us with more than 32).
__device__ __forceinline__ int i8_tile_rows(int m, int tile) {
    if (tile == 0) return 0;
    if (tile == 128) return m <= 64 ? 0 : m;
    const int tail = m % tile;
    return tail <= I8_GROUP ? m - tail : m;
}

// Four columns' sums of a row, scaled: s ws_e[n] acc, or s acc (SCALED: the output columns have scales).
template <bool SCALED>
__device__ __forceinline__ uint2 i8_scale4(int a0, int a1, int a2, int a3, float s, f32x4 c) {
    float y[4] = {static_cast<float>(a0) * s, static_cast<float>(a1) * s, static_cast<float>(a2) * s,
                  static_cast<float>(a3) * s};
    if constexpr (SCALED) {
#pragma unroll
        for (int x = 0; x < 4; ++x) y[x] *= c[x];
    }
    return make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
}

// One wave's 32 output columns (block nb) for up to 32 TB rows over the whole summed dimension, G steps of weights
// and rows loaded while G are multiplied.
template <int TB>
__device__ __forceinline__ void i8_stream_block(const Int8Params& p, const int8_t* w, const float* ws, int row0, int rows,
                                                int nb, int nsteps) {
    constexpr int G = TB == 1 ? 8 : (TB == 2 ? 4 : 2);
    const int lane = threadIdx.x & 63;
    const int8_t* wp = w + static_cast<int64_t>(nb) * nsteps * 1024 + lane * 16;
    const int8_t* tp[TB];
#pragma unroll
    for (int i = 0; i < TB; ++i)
        tp[i] = p.q + static_cast<int64_t>(row0 + min(i * 32 + (lane & 31), rows - 1)) * 64 + 16 * (lane >> 5);
    const int64_t block = static_cast<int64_t>(p.M) * 64;   // bytes of 64 columns of all rows
    i32x16 acc[TB];
#pragma unroll
    for (int i = 0; i < TB; ++i) acc[i] = i32x16{};
    i32x4 wv[2][G], tv[2][G][TB];
    auto load = [&](int buf, int g) {
#pragma unroll
        for (int u = 0; u < G; ++u) {
            const int st = min(g + u, nsteps - 1);
            wv[buf][u] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(wp + static_cast<int64_t>(st) * 1024));
#pragma unroll
            for (int i = 0; i < TB; ++i)
                tv[buf][u][i] = *reinterpret_cast<const i32x4*>(tp[i] + (st >> 1) * block + (st & 1) * 32);
        }
    };
    auto mma = [&](int buf, int g) {
#pragma unroll
        for (int u = 0; u < G; ++u)
            if (g + u < nsteps) {
#pragma unroll
                for (int i = 0; i < TB; ++i)
                    acc[i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wv[buf][u], tv[buf][u][i], acc[i], 0, 0, 0);
            }
    };
    load(0, 0);
    for (int g = 0; g < nsteps; g += 2 * G) {
        load(1, g + G);
        mma(0, g);
        load(0, g + 2 * G);
        mma(1, g + G);
    }
    // lane holds token lane & 31 of each 32-row block and, in register 4q + x, column 32 nb + 8q + 4(lane >> 5) + x
#pragma unroll
    for (int i = 0; i < TB; ++i) {
        const int r = i * 32 + (lane & 31);
        if (r >= rows) continue;
        const float sr = p.s[row0 + r];
        uint16_t* orow = p.out + static_cast<int64_t>(row0 + r) * p.N;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int n = nb * 32 + 8 * q + 4 * (lane >> 5);
            if (n >= p.N) continue;
            const f32x4 one = {1.0f, 1.0f, 1.0f, 1.0f};
            const f32x4 c = ws ? *reinterpret_cast<const f32x4*>(ws + n) : one;   // times one is exact
            *reinterpret_cast<uint2*>(orow + n) =
                i8_scale4<true>(acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3], sr, c);
        }
    }
}

// Column blocks [nb0, nb1) for up to 32 TB rows, dealt to the workgroup's four waves.  The
// rows' operands lie in `panel` (LDS, TB of 1 KiB a step).  The weights come as one
// stream over a wave's blocks, in units of four steps (the summed width is padded to
// that), all but one of R units ahead, the first of them from before the panel is filled: nothing drains at a
// block's end, where the sums are stored, and loads are repeated only at the stretch's own end.
template <int TB, bool SCALED>
__device__ __forceinline__ void i8_stream_blocks(const Int8Params& p, const int8_t* w, const float* ws, int row0, int rows,
                                                 int nb0, int nb1, int nsteps, int8_t* panel) {
    constexpr int W = 4, U = 4, R = 8;
    const int lane = threadIdx.x & 63, nu = nsteps / U;
    int nb = nb0 + uni(threadIdx.x >> 6);
    const int total = (nb1 - nb + W - 1) / W * nu;   // none for a wave without a block
    float sr[TB];
#pragma unroll
    for (int i = 0; i < TB; ++i) sr[i] = p.s[row0 + min(i * 32 + (lane & 31), rows - 1)];
    f32x4 cs[4];
    auto load_scales = [&](int b) {
        if constexpr (SCALED) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                cs[q] = *reinterpret_cast<const f32x4*>(ws + min(b * 32 + 8 * q + 4 * (lane >> 5), p.N - 4));
        }
    };
    load_scales(nb);
    const int8_t* lp = w + static_cast<int64_t>(min(nb, nb1 - 1)) * nsteps * 1024;
    int lk = 0, lf = 0;   // the next unit to load: of its block, and of all
    i32x4 wv[R][U];
    auto load = [&](i32x4(&v)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(lp + lane * 16 + u * 1024));
        const bool wrap = ++lk == nu;
        lk = wrap ? 0 : lk;
        if (++lf < total) lp += static_cast<int64_t>(U) * 1024 + (wrap ? static_cast<int64_t>(W - 1) * nsteps * 1024 : 0);
    };
    i32x16 acc[TB];
#pragma unroll
    for (int i = 0; i < TB; ++i) acc[i] = i32x16{};
    // in this order: the first unit's wait would otherwise be for all
#pragma unroll
    for (int i = 0; i < R - 1; ++i) {
        load(wv[i]);
        __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();   // the last panel is read
    constexpr int F = 8;   // loads of a thread in flight
    for (int i0 = threadIdx.x; i0 < nsteps * TB * 64; i0 += F * W * 64) {
        i32x4 v[F];
#pragma unroll
        for (int j = 0; j < F; ++j) {
            // operand bytes 16 i: of step st, row block b, row r % 32, columns 16 h onwards
            const int i = min(i0 + j * W * 64, nsteps * TB * 64 - 1);
            const int st = (i >> 6) / TB, r = ((i >> 6) % TB) * 32 + (i & 31), h = (i >> 5) & 1;
            v[j] = *reinterpret_cast<const i32x4*>(p.q + (static_cast<int64_t>(st >> 1) * p.M + row0 + min(r, rows - 1)) * 64 +
                                                   (st & 1) * 32 + 16 * h);
        }
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const int i = i0 + j * W * 64;
            if (i < nsteps * TB * 64) *reinterpret_cast<i32x4*>(panel + i * 16) = v[j];
        }
    }
    __syncthreads();
    int k = 0;
    for (int f = 0; f < total; f += R) {
        // the last round's units past the end multiply what was loaded last and are not stored
        static_for<R>([&](auto i_tag) {
            constexpr int at = decltype(i_tag)::value;
            load(wv[(at + R - 1) % R]);
            const int8_t* op = panel + k * (U * TB * 1024) + lane * 16;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < TB; ++i)
                    acc[i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
                        wv[at][u], *reinterpret_cast<const i32x4*>(op + (u * TB + i) * 1024), acc[i], 0, 0, 0);
            if (++k == nu) {
                k = 0;
#pragma unroll
                for (int i = 0; i < TB; ++i) {
                    const int r = i * 32 + (lane & 31);
                    uint16_t* orow = p.out + static_cast<int64_t>(row0 + r) * p.N;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int n = nb * 32 + 8 * q + 4 * (lane >> 5);
                        const uint2 y = i8_scale4<SCALED>(acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2],
                                                          acc[i][4 * q + 3], sr[i], cs[q]);
                        if (r < rows && n < p.N && nb < nb1) *reinterpret_cast<uint2*>(orow + n) = y;
                    }
                    acc[i] = i32x16{};
                }
                nb += W;
                load_scales(nb);
            }
        });
    }
}

// The list of all (row group, 32-column block) pairs, groups of p.group rows, by
// workgroups of four waves, a wave a block.  s_off, s_pre: [E + 1].
//
// PANEL: each workgroup takes an equal stretch of the list and keeps the rows
// of the group it is in in LDS in operand order (p.group is
// what 128 KiB hold of the summed width): read by every wave from memory they
// cost nearly as much of the load path as the weights (128 experts of 22 rows,
// K 2688, N 3712, quantization included: 294 us from memory, 245 us here, 5.6 TB/s in this kernel).
// Otherwise, for few rows in all and for wide ones: items of four blocks, a wave each, in turn.
template <bool PANEL, bool SCALED>
__device__ __forceinline__ void i8_stream_list(const Int8Params& p, int* s_off, int* s_pre, int8_t* s_panel) {
    constexpr int W = 4;
    const int nblocks = (p.N + 31) / 32, nsteps = p.width / 32;
    prefix_experts(p.offsets, p.E, p.M, s_off, s_pre,
                   [&](int m) { return (m - i8_tile_rows(m, p.tile) + p.group - 1) / p.group * nblocks; });
    const int64_t total = uni(s_pre[p.E]);
    const int wave = uni(threadIdx.x >> 6);
    // items of the list: one stretch a workgroup, or four blocks each
    const int64_t items = PANEL ? gridDim.x : (total + W - 1) / W;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        int at = static_cast<int>(total * it / items);
        const int end = static_cast<int>(total * (it + 1) / items);
        while (at < end) {   // one row group's part of the item
            const int e = uni(find_expert_wave(s_pre, p.E, at));
            const int local = at - uni(s_pre[e]), grp = local / nblocks, nb0 = local - grp * nblocks;
            const int nb1 = min(nblocks, nb0 + end - at);
            const int lo = uni(s_off[e]), hi = uni(s_off[e + 1]);
            const int row0 = lo + i8_tile_rows(hi - lo, p.tile) + grp * p.group;
            const int rows = min(p.group, hi - row0);
            const int8_t* w = p.w + static_cast<int64_t>(e) * p.w_stride;
            const float* ws = p.ws ? p.ws + static_cast<int64_t>(e) * p.ws_ld : nullptr;
            const int tb = (rows + 31) / 32;
            if constexpr (PANEL) {
                if (tb == 1) i8_stream_blocks<1, SCALED>(p, w, ws, row0, rows, nb0, nb1, nsteps, s_panel);
                else if (tb == 2) i8_stream_blocks<2, SCALED>(p, w, ws, row0, rows, nb0, nb1, nsteps, s_panel);
                else i8_stream_blocks<3, SCALED>(p, w, ws, row0, rows, nb0, nb1, nsteps, s_panel);
            } else {
                for (int nb = nb0 + wave; nb < nb1; nb += W) {
                    if (tb == 1) i8_stream_block<1>(p, w, ws, row0, rows, nb, nsteps);
                    else if (tb == 2) i8_stream_block<2>(p, w, ws, row0, rows, nb, nsteps);
                    else i8_stream_block<3>(p, w, ws, row0, rows, nb, nsteps);
                }
            }
            at += nb1 - nb0;
        }
    }
}

__global__ __launch_bounds__(256) void int8_stream_kernel(const Int8Params p) {
    __shared__ int s_off[GG_KMAX_EXPERTS + 1];
    __shared__ int s_pre[GG_KMAX_EXPERTS + 1];
    i8_stream_list<false, false>(p, s_off, s_pre, nullptr);
}

// Tiles: 64 B rows x 64 B output columns by four waves, each 32 B x 32 B, as
// B x B accumulators of 32 x 32.  B = 4 (256 x 256) fills the accumulation
// registers; B = 2 (128 x 128) gives four times the tiles where there would
// be fewer large ones than CUs (777 rows over 5 experts, K 1048, N 2056: 21 us, 30 us with B = 4).
// With B = 4 a tile costs about 0.83 us a stage and 8.6 us besides: 262144 rows, K = N = 4096, 3.9 ms, 2250
// TOP/s, what the chip's power leaves for random operands; 131072 rows, K 768, N 2048, 340 us, 1210 TOP/s in the tiles.
// Rows and weights stream into an LDS ring (128 KiB: four stages, or eight)
// of 64-byte stages by LDS-DMA, all but one of them ahead: the rows, 16-byte
// chunk c of row r at c ^ ((r >> 2) & 3), and the weights as they lie in
// the packed layout; fragment reads of both are free of bank conflicts.  Each
// of a stage's two 32-byte steps is B x B matrix instructions a wave, while the
// next step's 2 B fragments are read; the only barrier of a stage sits
// in its second step, where the next stage has landed and every wave has
// read the last fragments of this one, whose slot is refilled from there on.
// The epilogue scales and rounds through a small staging area of its own, so
// the next tile's first stages are already on their way, and the waits of
// those stages leave the epilogue's stores outstanding: memory operations
// complete in order, and the stores were issued after the copies.
constexpr int I8_STAGE = 64;
constexpr int I8_STG_BYTES = 32 * 128;   // per wave: 32 rows x 64 columns of bf16

__device__ __forceinline__ int acc_rd_i(int a) {
    int v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
    return v;
}

template <int B, bool SCALED>   // SCALED: the output columns have scales
__global__ __launch_bounds__(256, 1) void int8_tile_kernel(const Int8Params p) {
    constexpr int TILE = 64 * B;                            // rows, and columns
    constexpr int SLOT_BYTES = 2 * TILE * I8_STAGE, SLOTS = I8_RING / SLOT_BYTES;
    constexpr int P = 2 * B;                                // copies a wave issues for a stage
    __shared__ __attribute__((aligned(1024))) int8_t s_ring[I8_RING];
    __shared__ __attribute__((aligned(16))) int8_t s_stg[4 * I8_STG_BYTES];
    __shared__ int s_off[GG_KMAX_EXPERTS + 1];
    __shared__ int s_pre[GG_KMAX_EXPERTS + 1];
    const int nblocks = (p.N + 31) / 32, nsteps = p.width / 32, nstages = p.width / I8_STAGE;
    const int tiles_n = (p.N + TILE - 1) / TILE;
    prefix_experts(p.offsets, p.E, p.M, s_off, s_pre,
                   [&](int m) { return (i8_tile_rows(m, TILE) + TILE - 1) / TILE * tiles_n; });
    const int n_tiles = uni(s_pre[p.E]);
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int wr = wave >> 1, wc = wave & 1;      // the wave's rows and columns
    // consecutive tiles to the workgroups of one XCD, which share an L2
    const int G = gridDim.x, b = blockIdx.x;
    const int slot = (G % 8 == 0) ? (b & 7) * (G >> 3) + (b >> 3) : b;
    const uint32_t ring = lds_addr(s_ring);

    // what the copies of one tile read
    const int8_t* t_base = nullptr;   // its first row
    const int8_t* w_base = nullptr;   // its expert's matrix
    uint32_t t_voff[B];               // this lane's chunks of rows 16 B wave + 16 i ..
    int wb[B / 2];                    // this wave's 32-column blocks
    const int64_t t_block = static_cast<int64_t>(p.M) * I8_STAGE;   // bytes of 64 columns of all rows
    int e = 0, row0 = 0, rows = 0, col0 = 0;
    auto setup = [&](int t) {
        e = uni(find_expert_wave(s_pre, p.E, t));
        const int local = t - uni(s_pre[e]);
        const int lo = uni(s_off[e]), m = i8_tile_rows(uni(s_off[e + 1]) - lo, TILE);
        const int tiles_m = (m + TILE - 1) / TILE;
        const int tm = local % tiles_m, tn = local / tiles_m;
        row0 = lo + tm * TILE;
        rows = min(TILE, m - tm * TILE);
        col0 = tn * TILE;
        t_base = p.q + static_cast<int64_t>(row0) * I8_STAGE;
        w_base = p.w + static_cast<int64_t>(e) * p.w_stride;
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int r = 16 * B * wave + 16 * i + (lane >> 2);
            const int c = (lane & 3) ^ ((r >> 2) & 3);
            t_voff[i] = static_cast<uint32_t>(min(r, rows - 1)) * I8_STAGE + 16 * c;
        }
#pragma unroll
        for (int i = 0; i < B / 2; ++i) wb[i] = min(col0 / 32 + B / 2 * wave + i, nblocks - 1);
    };
    // One of the P copies of a stage that this wave issues (nothing past the last stage).
    auto piece = [&](int st, auto i_tag) {
        constexpr int i = decltype(i_tag)::value;
        if (st >= nstages) return;
        const uint32_t dst = ring + (st & (SLOTS - 1)) * SLOT_BYTES;
        if constexpr (i < B) {
            dma16(t_base + st * t_block, t_voff[i], dst + (16 * B * wave + 16 * i) * I8_STAGE);
        } else {
            constexpr int h = (i - B) >> 1, u = i & 1;
            dma16(w_base + (static_cast<int64_t>(wb[h]) * nsteps + 2 * st + u) * 1024, lane * 16,
                  dst + TILE * I8_STAGE + ((B / 2 * wave + h) * 2 + u) * 1024);
        }
    };

    i32x16 acc[B][B];    // [row block][column block]
    i32x4 tf[2][B], wf[2][B];
    auto read_t = [&](int st, auto u_tag) {
        constexpr int u = decltype(u_tag)::value;
        const int8_t* sl = s_ring + (st & (SLOTS - 1)) * SLOT_BYTES;
        const int c = (2 * u + (lane >> 5)) ^ ((lane >> 2) & 3);
#pragma unroll
        for (int i = 0; i < B; ++i)
            tf[u][i] = *reinterpret_cast<const i32x4*>(sl + (32 * B * wr + 32 * i + (lane & 31)) * I8_STAGE + 16 * c);
    };
    auto read_w = [&](int st, auto u_tag) {
        constexpr int u = decltype(u_tag)::value;
        const int8_t* sl = s_ring + (st & (SLOTS - 1)) * SLOT_BYTES;
#pragma unroll
        for (int j = 0; j < B; ++j)
            wf[u][j] = *reinterpret_cast<const i32x4*>(sl + TILE * I8_STAGE + ((B * wc + j) * 2 + u) * 1024 + lane * 16);
    };
    // the B matrix instructions of row block i in step u; the tile's first step starts its sums from zero
    auto mma = [&](auto u_tag, auto i_tag, auto first_tag) {
        constexpr int u = decltype(u_tag)::value, i = decltype(i_tag)::value;
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if constexpr (decltype(first_tag)::value != 0)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[u][j], tf[u][i], i32x16{}, 0, 0, 0);
            else
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[u][j], tf[u][i], acc[i][j], 0, 0, 0);
        }
    };
    auto fence = [&]() { __builtin_amdgcn_sched_barrier(0); };
    // Waits until at most n copies and stores issued after those of the stage that is needed are outstanding.
    auto wait_after = [&](int n) {
        if (n >= 60) wait_vmcnt<60>();
        else if (n >= 52) wait_vmcnt<52>();
        else if (n >= 44) wait_vmcnt<44>();
        else if (n >= 36) wait_vmcnt<36>();
        else if (n >= 28) wait_vmcnt<28>();
        else if (n >= 24) wait_vmcnt<24>();
        else if (n >= 20) wait_vmcnt<20>();
        else if (n >= 16) wait_vmcnt<16>();
        else if (n >= 12) wait_vmcnt<12>();
        else if (n >= 8) wait_vmcnt<8>();
        else if (n >= 4) wait_vmcnt<4>();
        else wait_vmcnt<0>();
    };
    // Stage st: two steps of B groups of B matrix instructions, each group
    // followed by one copy; the next step's fragments are read during the
    // first groups of a step.  behind: the stores and loads issued behind the
    // copies of the prologue's stages, at least.
    auto stage = [&](int st, int behind, auto first_tag, auto last_tag) {
        const int c1 = decltype(first_tag)::value != 0 ? nstages : st + SLOTS - 1;    // the prologue brought that stage
        static_for<B>([&](auto it) {
            constexpr int i = decltype(it)::value;
            if constexpr (i == 0) read_w(st, GrpTag<1>{});
            if constexpr (i == 1) read_t(st, GrpTag<1>{});
            mma(GrpTag<0>{}, it, first_tag);
            piece(c1, GrpTag<B - 1 + i>{});
            fence();
        });
        mma(GrpTag<1>{}, GrpTag<0>{}, GrpTag<0>{});
        piece(c1, GrpTag<P - 1>{});
        fence();
        if constexpr (decltype(last_tag)::value == 0) {
            // stage st + 1 has landed, and every wave holds its last fragments of stage st, whose slot
            // is refilled from here on
            wait_after(P * min(nstages - 2 - st, SLOTS - 2) + (st < SLOTS - 1 ? behind : 0));
            block_barrier();
        }
        static_for<B - 1>([&](auto it) {
            constexpr int i = decltype(it)::value;
            if constexpr (decltype(last_tag)::value == 0) {
                if constexpr (i == 0) read_w(st + 1, GrpTag<0>{});
                if constexpr (i == (B > 2 ? 1 : 0)) read_t(st + 1, GrpTag<0>{});
            }
            mma(GrpTag<1>{}, GrpTag<i + 1>{}, GrpTag<0>{});
            if constexpr (decltype(last_tag)::value == 0) piece(st + SLOTS, it);
            fence();
        });
    };
    constexpr int SCALE_LOADS = SCALED ? B + 4 * B : B;
    // the copies before a tile's first stage: the whole ring's
    auto prologue = [&]() {
        for (int st = 0; st < SLOTS; ++st) static_for<P>([&](auto i) { piece(st, i); });
    };

    int t = slot, stores = 0;
    if (t < n_tiles) {
        setup(t);
        prologue();
    }
    while (t < n_tiles) {
        wait_after(P * min(nstages - 1, SLOTS - 1) + stores);        // stage 0
        block_barrier();
        // the scales of this tile, for its epilogue: lane holds, of
        // block (i, j), row 32 i + (lane & 31) and columns 32 j + 8 q + 4 (lane >> 5) .. + 3
        const int prow0 = row0, prows = rows, gc0 = col0 + 32 * B * wc;
        float sr[B];
        f32x4 cs[SCALED ? B : 1][4];
#pragma unroll
        for (int i = 0; i < B; ++i) sr[i] = p.s[row0 + min(32 * B * wr + 32 * i + (lane & 31), rows - 1)];
        if constexpr (SCALED) {
            const float* ws = p.ws + static_cast<int64_t>(e) * p.ws_ld;
#pragma unroll
            for (int j = 0; j < B; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    cs[j][q] = *reinterpret_cast<const f32x4*>(ws + min(gc0 + 32 * j + 8 * q + 4 * (lane >> 5), p.N - 4));
        }
        const int behind = stores + SCALE_LOADS;
        read_w(0, GrpTag<0>{});
        read_t(0, GrpTag<0>{});
        stage(0, behind, GrpTag<1>{}, GrpTag<0>{});
        for (int st = 1; st < nstages - 1; ++st) stage(st, behind, GrpTag<0>{}, GrpTag<0>{});
        stage(nstages - 1, behind, GrpTag<0>{}, GrpTag<1>{});
        t += G;
        wait_vmcnt<0>();         // the scales
        // held from here on, so that nothing waits for them behind the next tile's copies
#pragma unroll
        for (int i = 0; i < B; ++i) {
            asm volatile("" : "+v"(sr[i]));
            if constexpr (SCALED) {
#pragma unroll
                for (int q = 0; q < 4; ++q) asm volatile("" : "+v"(cs[i][q]));
            }
        }
        block_barrier();         // and every wave is done with the ring
        if (t < n_tiles) {
            setup(t);
            prologue();
        }
        // All stores of a wave are issued where the tile is full; a store whose lanes all lie outside may be
        // skipped, so a partial tile counts as none.
        stores = prows == TILE && gc0 - 32 * B * wc + TILE <= p.N ? 2 * B * B : 0;
        mfma_drain();
        int opaque = 0;
        asm volatile("" : "+s"(opaque));
        const int ln = lane + opaque;
        uint16_t* stg = reinterpret_cast<uint16_t*>(s_stg + wave * I8_STG_BYTES) + opaque;
        // B * B / 2 blocks of 32 rows x 64 columns go through the staging area, [32 rows][64 columns] with 16-byte
        // chunk c of row r at c ^ (r & 7); the arithmetic of a block covers the LDS round trip of the last.
        auto scaled = [&](auto b_tag, uint2 (&v)[8]) {
            constexpr int i = decltype(b_tag)::value % B, jh = decltype(b_tag)::value / B;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int j = 2 * jh + (c >> 2), q = c & 3;
                const i32x16& a = acc[i][j];
                float y[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    y[x] = static_cast<float>(acc_rd_i(a[4 * q + x])) * sr[i];
                    if constexpr (SCALED) y[x] *= cs[j][q][x];
                }
                v[c] = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
            }
        };
        auto put = [&](const uint2 (&v)[8]) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int rr = ln & 31;
                *reinterpret_cast<uint2*>(stg + rr * 64 + ((c ^ (rr & 7)) << 3) + 4 * (ln >> 5)) = v[c];
            }
        };
        uint2 vals[8];
        scaled(GrpTag<0>{}, vals);
        put(vals);
        static_for<B * B / 2>([&](auto b_tag) {
            constexpr int b = decltype(b_tag)::value, i = b % B, jh = b / B;
            if constexpr (b < B * B / 2 - 1) scaled(GrpTag<b + 1>{}, vals);
            uint4 out[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                out[k] = *reinterpret_cast<const uint4*>(stg + (8 * k + (ln >> 3)) * 64 + (ln & 7) * 8);
            if constexpr (b < B * B / 2 - 1) put(vals);
            // lane: row 8 k + (ln >> 3), 16-byte chunk (ln & 7) ^ (ln >> 3)
            const int gc = gc0 + 64 * jh + 8 * ((ln & 7) ^ (ln >> 3)), gr = 32 * B * wr + 32 * i + (ln >> 3);
            uint16_t* to = p.out + static_cast<int64_t>(prow0 + gr) * p.N + gc;
            if (stores) {
#pragma unroll
                for (int k = 0; k < 4; ++k) st16_nt(to + static_cast<int64_t>(8 * k) * p.N, out[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (gr + 8 * k < prows && gc < p.N) st16_nt(to + static_cast<int64_t>(8 * k) * p.N, out[k]);
            }
        });
    }
    if (p.group == 0) return;   // another launch's
    __syncthreads();
    i8_stream_list<true, SCALED>(p, s_off, s_pre, s_ring);
}

// ---------------------------------------------------------------- launchers
template <int MODE, int Y>
static hipError_t launch_quant(const QuantParams& p, int num_cu, hipStream_t s) {
    const int units = p.K / (8 * QuantUnit<MODE>::HALVES);
    // four waves a workgroup; pairs of rows start at an even one
    const int64_t want = (static_cast<int64_t>(p.M) / Y + 1 + 3) / 4, most = static_cast<int64_t>(num_cu) * 16;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most)), block(256);
    if (units <= 64) hipLaunchKernelGGL((quant_rows_kernel<MODE, 1, Y>), grid, block, 0, s, p);
    else if (units <= 128) hipLaunchKernelGGL((quant_rows_kernel<MODE, 2, Y>), grid, block, 0, s, p);
    else if (units <= 256) hipLaunchKernelGGL((quant_rows_kernel<MODE, 4, Y>), grid, block, 0, s, p);
    else if (units <= 512 && MODE != Q_DGLU)
        hipLaunchKernelGGL((quant_rows_kernel<MODE, MODE == Q_DGLU ? 4 : 8, Y>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((quant_rows_kernel<MODE, 0, Y>), grid, block, 0, s, p);
    return hipGetLastError();
}

hipError_t launch_quant_rows(QuantMode mode, const QuantParams& p, int num_cu, hipStream_t s) {
    if (p.M <= 0) return hipSuccess;
    // pairs where they leave at least eight waves for each CU
    const bool pairs = p.blocked && p.M >= 16 * num_cu;
    switch (mode) {
        case Q_PLAIN: return pairs ? launch_quant<Q_PLAIN, 2>(p, num_cu, s) : launch_quant<Q_PLAIN, 1>(p, num_cu, s);
        case Q_GLU: return pairs ? launch_quant<Q_GLU, 2>(p, num_cu, s) : launch_quant<Q_GLU, 1>(p, num_cu, s);
        case Q_SCALED: return launch_quant<Q_SCALED, 1>(p, num_cu, s);
        default: return launch_quant<Q_DGLU, 1>(p, num_cu, s);
    }
}

hipError_t launch_int8_pack(const int8_t* q, const float* s, int E, int N, int K, int transposed, int8_t* packed,
                            hipStream_t stream) {
    const int64_t rows = i8_rows_p(transposed ? K : N), cont = i8_cont_p(transposed ? N : K);
    const int64_t bytes = E * rows * cont;
    int64_t blocks = (bytes / 16 + 255) / 256;
    if (blocks > 65536) blocks = 65536;
    hipLaunchKernelGGL(int8_pack_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, q, s, E, N, K,
                       transposed, packed, reinterpret_cast<float*>(packed + bytes), static_cast<int>(i8_cont_p(N)));
    return hipGetLastError();
}

template <int B>
static hipError_t launch_tiles(const Int8Params& p, int num_cu, hipStream_t s) {
    constexpr int TILE = 64 * B;
    const int64_t upper = (static_cast<int64_t>(p.M) / TILE + (p.M < p.E ? p.M : p.E)) * ((p.N + TILE - 1) / TILE);
    const dim3 grid(static_cast<unsigned>(upper < num_cu && p.group == 0 ? upper : num_cu));
    if (p.ws) hipLaunchKernelGGL((int8_tile_kernel<B, true>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((int8_tile_kernel<B, false>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_int8_gemm(const Int8Params& p, int num_cu, hipStream_t s) {
    Int8Params g = p;
    const Int8Plan plan = i8_plan(p.M, p.E, p.N, p.width, num_cu);
    g.tile = plan.tile;
    g.group = plan.group;
    if (g.tile) {
        const hipError_t st = g.tile == 256 ? launch_tiles<4>(g, num_cu, s) : launch_tiles<2>(g, num_cu, s);
        if (st != hipSuccess || g.group) return st;
    }
    g.group = I8_GROUP;
    const int64_t nblocks = (p.N + 31) / 32;
    const int64_t groups = static_cast<int64_t>(p.M) / I8_GROUP + (p.M < p.E ? p.M : p.E);
    const int64_t upper = (groups * nblocks + 3) / 4, most = static_cast<int64_t>(num_cu) * 3;
    hipLaunchKernelGGL(int8_stream_kernel, dim3(static_cast<unsigned>(upper < most ? upper : most)), dim3(256), 0, s, g);
    return hipGetLastError();
}

}  // namespace gg
