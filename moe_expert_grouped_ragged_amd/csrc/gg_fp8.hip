// Expert products in 8-bit floating point on CDNA4: quantization in blocks of
// 128 (with the activation or its derivative fused in), the packed weight
// layout, and the ragged grouped product on the block-scaled matrix instruction.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gg_device.h"
#include "gg_fp8.h"
#include "gg_kernels.h"

namespace gg {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;

// ---------------------------------------------------------------- quantization
//
// A block of 128 values has one power of two, 2^c, the least (c >= -126) with
// max|v| <= 448 * 2^c; q = v / 2^c rounded to nearest even in e4m3.  The
// division is exact (down to fp32's subnormals, which round to zero in e4m3),
// so q is what the definition says, bit for bit, and 448 is never passed.  With
// max|v| = m 2^x, 1 <= m < 2: c = x - 8, or x - 7 where m > 1.75.  A block that
// holds a NaN or an infinity becomes NaNs (0x7f).
struct F8Scale {
    float inv;       // 2^-c
    uint32_t byte;   // c + 127
    bool nan;
};
// top: the largest |v| of the block as fp32 bits
__device__ __forceinline__ F8Scale f8_scale(uint32_t top) {
    F8Scale s;
    int c = static_cast<int>((top + 0x1fffffu) >> 23) - 8;   // c + 127: m > 1.75 carries into the exponent
    s.nan = top >= 0x7f800000u;
    c = max(c, 1);
    c = s.nan ? 127 : c;
    s.byte = static_cast<uint32_t>(c);
    s.inv = __builtin_bit_cast(float, static_cast<uint32_t>(254 - c) << 23);
    return s;
}
// Four values to four e4m3 bytes.
__device__ __forceinline__ uint32_t f8_four(float a, float b, float c, float d, const F8Scale& s) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * s.inv, b * s.inv, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c * s.inv, d * s.inv, r, true);
    return s.nan ? 0x7f7f7f7fu : static_cast<uint32_t>(r);
}
// Running |v| maxima of packed pairs of bf16 values, half by half, and the larger half as fp32 bits.
__device__ __forceinline__ uint32_t f8_max2(uint32_t top, uint32_t pair) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, top),
                                                                  __builtin_bit_cast(u16x2, pair & 0x7fff7fffu)));
}
__device__ __forceinline__ uint32_t f8_top(uint32_t top) { return max(top << 16, top & 0xffff0000u); }
// The largest of the values of 16 neighbouring lanes (a row of the data-parallel moves): lanes ^ 1, ^ 2, then the other
// four, the other eight.
__device__ __forceinline__ uint32_t f8_top16(uint32_t m) {
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0xb1, 0xf, 0xf, true)));
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x4e, 0xf, 0xf, true)));
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x141, 0xf, 0xf, true)));
    return max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x140, 0xf, 0xf, true)));
}

// The activation and its derivative on bf16 values: A = bf16(act(gate) * up), dH1 = bf16 of dg and du.  e: -slope
// log2 e, so that the sigmoid is one product, 2^x, a sum and a reciprocal.
__device__ __forceinline__ float f8_log2e(float slope) { return -1.44269504088896340736f * slope; }
__device__ __forceinline__ float f8_sigmoid(float g, float e) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(e * g));
}
__device__ __forceinline__ float f8_act(float g, float u, float e) { return g * f8_sigmoid(g, e) * u; }
__device__ __forceinline__ void f8_act_grad(float g, float u, float da, float slope, float e, float& dg, float& du) {
    const float sg = f8_sigmoid(g, e), t = da * sg;
    dg = t * u * (1.0f + slope * g * (1.0f - sg));
    du = t * g;
}

// A wave takes 512 columns of two neighbouring rows, from an even one on: 8 columns of each a lane, so 16 lanes are a
// block and its maximum stays in registers.  Pairs of lanes then exchange halves, so that a store is 16 bytes a lane and
// whole 128-byte lines of the two rows in the product's layout (262144 x 4096, 3.2 GB: 575 us, 5.6 TB/s; 665 us with 16
// columns of one row a lane, whose stores are half lines).  A block needs no more of its row, so a row is a wave's or
// several's and the values are never held beyond their block.  U such groups of columns are in flight at a time (four
// and, with the activation, two: 640 us with two; a single one for few rows, for more waves).  Bound by the bytes.
template <int MODE, int U>
__global__ __launch_bounds__(256) void f8_quant_kernel(const F8QuantParams p) {
    constexpr int PARTS = MODE == F8_DGLU ? 2 : 1;    // blocks that a lane makes at a time
    constexpr int IN = MODE == F8_PLAIN ? 1 : (MODE == F8_GLU ? 2 : 3);
    const int lane = threadIdx.x & 63;
    const auto clamp = [&](int64_t o) { return static_cast<int>(o < 0 ? 0 : (o > p.M ? p.M : o)); };
    const int lo = clamp(p.offsets[0]), hi = clamp(p.offsets[p.E]);
    const int part = p.dim.part, part_p = p.dim.part_p;
    const int width = MODE == F8_DGLU ? part_p : p.dim.padded();
    const int64_t qblock = static_cast<int64_t>(p.M) * 64;
    const float e2 = f8_log2e(p.slope);
    const int c0 = static_cast<int>(blockIdx.y) * U * 512 + 8 * lane;
    if (lo >= hi) return;      // also where lo is odd
    for (int64_t r0 = (lo & ~1) + 2 * (static_cast<int64_t>(blockIdx.x) * 4 + uni(threadIdx.x >> 6)); r0 < hi;
         r0 += static_cast<int64_t>(gridDim.x) * 8) {
        // rows that exist, where the pair has only one
        const int64_t row[2] = {r0 < lo ? r0 + 1 : r0, r0 + 1 < hi ? r0 + 1 : r0};
        uint4 in[U][2][IN];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 512, h = MODE != F8_DGLU && c >= part_p, k = c - h * part_p;
            const bool ok = c < width && k < part;
            const int col = ok ? h * part + k : 0;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint4 zero = make_uint4(0, 0, 0, 0);
                if constexpr (MODE == F8_PLAIN) {
                    in[u][y][0] = ok ? ld16_nt(p.x + row[y] * p.dim.real() + col) : zero;
                } else {
                    const uint16_t* g = (MODE == F8_GLU ? p.x : p.h1) + row[y] * 2 * part + col;
                    in[u][y][0] = ok ? ld16_nt(g) : zero;
                    in[u][y][1] = ok ? ld16_nt(g + part) : zero;
                    if constexpr (MODE == F8_DGLU) in[u][y][IN - 1] = ok ? ld16_nt(p.x + row[y] * part + col) : zero;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 512;
            if (c >= width) continue;     // whole blocks of lanes
            const int h = MODE != F8_DGLU && c >= part_p, k = c - h * part_p;
            uint2 q[PARTS][2];
            uint32_t byte[PARTS][2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t v[PARTS][4];         // 8 bf16 values
                const uint4(&x)[IN] = in[u][y];
                const uint32_t a[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
                const uint32_t b[4] = {x[IN > 1].x, x[IN > 1].y, x[IN > 1].z, x[IN > 1].w};
                const uint32_t d[4] = {x[IN - 1].x, x[IN - 1].y, x[IN - 1].z, x[IN - 1].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (MODE == F8_PLAIN) {
                        v[0][i] = a[i];
                    } else if constexpr (MODE == F8_GLU) {
                        v[0][i] = pack2(f8_act(lo_f(a[i]), lo_f(b[i]), e2), f8_act(hi_f(a[i]), hi_f(b[i]), e2));
                    } else {
                        float g0, u0, g1, u1;
                        f8_act_grad(lo_f(a[i]), lo_f(b[i]), lo_f(d[i]), p.slope, e2, g0, u0);
                        f8_act_grad(hi_f(a[i]), hi_f(b[i]), hi_f(d[i]), p.slope, e2, g1, u1);
                        v[0][i] = pack2(g0, g1);
                        v[PARTS - 1][i] = pack2(u0, u1);
                    }
                }
                if constexpr (MODE != F8_PLAIN) {
                    if (p.v_out && k < part) {      // twice the same where the pair has one row
                        uint16_t* o = p.v_out + row[y] * p.dim.real() + k;
#pragma unroll
                        for (int z = 0; z < PARTS; ++z) st16_nt(o + z * part, make_uint4(v[z][0], v[z][1], v[z][2], v[z][3]));
                    }
                }
#pragma unroll
                for (int z = 0; z < PARTS; ++z) {
                    const F8Scale s = f8_scale(f8_top16(f8_top(f8_max2(f8_max2(f8_max2(f8_max2(0, v[z][0]), v[z][1]), v[z][2]), v[z][3]))));
                    q[z][y] = make_uint2(f8_four(lo_f(v[z][0]), hi_f(v[z][0]), lo_f(v[z][1]), hi_f(v[z][1]), s),
                                         f8_four(lo_f(v[z][2]), hi_f(v[z][2]), lo_f(v[z][3]), hi_f(v[z][3]), s));
                    byte[z][y] = s.byte;
                }
            }
            // even lanes: 16 columns of the first row; odd lanes: of the second
            const bool odd = lane & 1;
            const int64_t r = r0 + odd;
            const bool live = r >= lo && r < hi;
#pragma unroll
            for (int z = 0; z < PARTS; ++z) {
                const uint2 send = odd ? q[z][0] : q[z][1], keep = odd ? q[z][1] : q[z][0];
                const uint2 got = make_uint2(__builtin_amdgcn_mov_dpp(send.x, 0xb1, 0xf, 0xf, true),
                                             __builtin_amdgcn_mov_dpp(send.y, 0xb1, 0xf, 0xf, true));
                // by bits: an index would put the two into memory
                const uint32_t mine = byte[z][0] ^ ((byte[z][0] ^ byte[z][1]) & (0u - static_cast<uint32_t>(odd)));
                if (!live) continue;
                const int cp = (c & ~15) + z * part_p, kb = cp / F8_BLOCK;
                *reinterpret_cast<uint4*>(p.q + (cp >> 6) * qblock + r * 64 + (cp & 63)) =
                    odd ? make_uint4(got.x, got.y, keep.x, keep.y) : make_uint4(keep.x, keep.y, got.x, got.y);
                if ((lane & 14) == 0)
                    p.s[4 * (static_cast<int64_t>(kb >> 2) * p.M + r) + (kb & 3)] = static_cast<uint8_t>(mine);
            }
        }
    }
}

// A workgroup a 128 x 128 block: 16 rows of 16 lanes of eight columns at a time, held in registers.  The grid has a row
// for each expert: a dimension of it holds less than 2^32 threads, 2^24 blocks (34 GB of weights 8 rows high).
__global__ __launch_bounds__(256) void f8_quant_weights_kernel(const uint16_t* __restrict__ w, F8Dim n, F8Dim k,
                                                               uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
    __shared__ uint32_t s_top[4];
    const int64_t b = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
    const int kb = static_cast<int>(b % k.blocks());
    const int64_t nb = b / k.blocks();                  // over all experts
    const int per = n.part_p / F8_BLOCK;                // blocks of a part; the parts of all experts follow each other
    const int64_t row0 = nb / per * n.part + nb % per * F8_BLOCK;
    const int rows = min(F8_BLOCK, n.part - static_cast<int>(nb % per) * F8_BLOCK);
    const int col = kb * F8_BLOCK + 8 * (threadIdx.x & 15), t = threadIdx.x >> 4;
    uint4 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (16 * i + t < rows && col < k.part) v[i] = *reinterpret_cast<const uint4*>(w + (row0 + 16 * i + t) * k.part + col);
        m = f8_max2(f8_max2(f8_max2(f8_max2(m, v[i].x), v[i].y), v[i].z), v[i].w);
    }
    m = f8_top(m);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d, 64)));
    if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = m;
    __syncthreads();
    const F8Scale sc = f8_scale(max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3])));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (16 * i + t >= rows || col >= k.part) continue;
        *reinterpret_cast<uint2*>(q + (row0 + 16 * i + t) * k.part + col) =
            make_uint2(f8_four(lo_f(v[i].x), hi_f(v[i].x), lo_f(v[i].y), hi_f(v[i].y), sc),
                       f8_four(lo_f(v[i].z), hi_f(v[i].z), lo_f(v[i].w), hi_f(v[i].w), sc));
    }
    if (threadIdx.x == 0) s[b] = static_cast<uint8_t>(sc.byte);
}

// ---------------------------------------------------------------- packing
// The real index of padded index i of a dimension, or -1.
__device__ __forceinline__ int f8_real(const F8Dim& d, int i) {
    const int h = i / d.part_p, k = i - h * d.part_p;
    return k < d.part ? h * d.part + k : -1;
}

__global__ void f8_pack_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, int E, F8Dim n, F8Dim k,
                               int transposed, uint8_t* __restrict__ packed, uint8_t* __restrict__ scales) {
    const F8Dim rows = transposed ? k : n, cont = transposed ? n : k;
    const int64_t nb = rows.padded() / 32, steps = cont.padded() / 64;
    const int64_t total = static_cast<int64_t>(E) * nb * steps * 128;   // 16-byte operands
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int K = k.real();
    for (int64_t i = first; i < total; i += stride) {
        const int l = static_cast<int>(i & 63), h = static_cast<int>(i >> 6) & 1;
        const int64_t blk = i >> 7;
        const int st = static_cast<int>(blk % steps), b = static_cast<int>(blk / steps % nb);
        const uint8_t* m = q + blk / steps / nb * n.real() * K;
        const int row = f8_real(rows, b * 32 + (l & 31));
        uint32_t w[4] = {0, 0, 0, 0};
        if (row >= 0) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {      // parts are multiples of 8: eights exist or do not
                const int c = f8_real(cont, st * 64 + 32 * (l >> 5) + 16 * h + 8 * y);
                if (c < 0) continue;
                if (transposed) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        w[2 * y + (j >> 2)] |= static_cast<uint32_t>(m[static_cast<int64_t>(c + j) * K + row]) << (8 * (j & 3));
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(m + static_cast<int64_t>(row) * K + c);
                    w[2 * y] = x.x;
                    w[2 * y + 1] = x.y;
                }
            }
        }
        *reinterpret_cast<uint4*>(packed + i * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    const int ld = f8_scale_ld(cont), rb = rows.blocks(), cb = cont.blocks();
    const int64_t count = static_cast<int64_t>(E) * rb * ld;
    for (int64_t i = first; i < count; i += stride) {
        const int c = static_cast<int>(i % ld), r = static_cast<int>(i / ld % rb);
        const int64_t e = i / ld / rb;
        scales[i] = c >= cb ? 0 : (transposed ? s[(e * cb + c) * rb + r] : s[(e * rb + r) * cb + c]);
    }
}

// ---------------------------------------------------------------- product
//
// out[r][n] = sum over blocks of 128 of 2^(s_r + s_w) sum q w, in one of two
// ways of summing.  Either way a kernel adds a row's products in the same order
// (steps of 64 columns), so a row's bits do not depend on the batch.
//
// The scaled instruction (F8Params::fp32_sums = 0) multiplies by both scales, so
// the sums run over all blocks without a step between them.  It adds eight
// neighbouring products at a time, each cut towards zero below 2^-13 of the power
// of two of the largest's factors, and joins these sums in fp32 (found with
// planted values; the 8-bit instructions without scales cut at the same place).
// On normal data that costs about 2^-13 of the result, next to the result's
// rounding to bf16, up to 2^-8: enough for a result that ends there.  Where the
// result is quantized again it is not: 1.5% of H1 round to another bf16 value, and
// of 768 values of A one or two a row to their neighbour in e4m3, which moves all
// of that row of y by up to 0.7% of its norm.
//
// With fp32 sums (fp32_sums = 1) both operands become bf16 values in registers,
// times their scales, and the bf16 instruction multiplies them: e4m3 has four
// significant bits, so value and product are exact, and the sums are fp32's (a
// product of 2^-24 of the largest is kept, 2^-26 is not).  Rows take half of
// their scale and weights twice theirs: a row's largest values times their scale
// round to 2^128, which bf16 does not hold.
__device__ __forceinline__ f32x16 f8_mma(i32x8 w, i32x8 t, f32x16 acc, int ws, int ts) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, t, acc, 0, 0, 0, ws, 0, ts);
}
typedef __attribute__((ext_vector_type(4))) uint32_t f8_bf16x8;     // eight bf16 values
__device__ __forceinline__ f32x16 f8_mma_bf16(f8_bf16x8 w, f8_bf16x8 t, f32x16 acc) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, t), acc, 0, 0, 0);
}
__device__ __forceinline__ float f8_row_factor(int byte) { return __builtin_bit_cast(float, static_cast<uint32_t>(byte - 1) << 23); }
__device__ __forceinline__ float f8_weight_factor(uint32_t byte) { return __builtin_bit_cast(float, min(byte + 1, 255u) << 23); }
// Eights: the values 8 S to 8 S + 7 of a lane's 32, which one 16-column instruction takes (any 16 columns do, as long as
// both operands have the same: those and the other half of the lanes').  Pair P of them, times a power of two.
template <int S, int P>
__device__ __forceinline__ void f8_pair(f8_bf16x8& v, i32x8 raw, float factor) {
    v[P] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<uint32_t>(raw[2 * S + P / 2]), factor, P % 2 != 0));
}
template <int S>
__device__ __forceinline__ f8_bf16x8 f8_eight(i32x8 raw, float factor) {
    f8_bf16x8 v;
    static_for<4>([&](auto p) { f8_pair<S, decltype(p)::value>(v, raw, factor); });
    return v;
}
__device__ __forceinline__ i32x8 f8_join(i32x4 a, i32x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// One wave-wide copy of 4 bytes a lane to LDS, as dma16.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma4(const void* base, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dword %0, %1"
                 :: "v"(voff), "s"(uni_ptr(base)), "s"(uni(lds)) : "memory", "m0");
}
#pragma clang diagnostic pop

// dma16 with AT bytes added to both addresses by the instruction.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int AT>
__device__ __forceinline__ void dma16_at(const void* base, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1 offset:%3"
                 :: "v"(voff), "s"(uni_ptr(base)), "s"(uni(lds)), "i"(AT) : "memory", "m0");
}
#pragma clang diagnostic pop

// A dword that no kernel of the launch writes, by the scalar unit.
__device__ __forceinline__ uint32_t scalar_load(const uint8_t* p) {
    return *(const __attribute__((address_space(4))) uint32_t*)(reinterpret_cast<uintptr_t>(uni_ptr(p)));
}

__device__ __forceinline__ uint32_t max_other_half(uint32_t v) {   // of lanes l and l ^ 32
    return max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 32, 64)));
}

// The panel of quantized rows, F 16-byte operands of a thread in flight.
template <int TB>
__device__ __forceinline__ void f8_copy_panel(const F8Params& p, int row0, int rows, uint8_t* panel, uint8_t* pscale) {
    constexpr int F = 8, T = 256;
    const int nu = p.kblocks, chunks = nu * TB * 256;
    for (int i0 = threadIdx.x; i0 < chunks; i0 += F * T) {
        i32x4 v[F];
#pragma unroll
        for (int j = 0; j < F; ++j) {
            // operand bytes 16 i: of step st, row block b, half h of 32 columns, lane l
            const int i = min(i0 + j * T, chunks - 1);
            const int l = i & 63, h = (i >> 6) & 1, st = (i >> 7) / TB, b = (i >> 7) % TB, r = b * 32 + (l & 31);
            if (r < rows)
                v[j] = *reinterpret_cast<const i32x4*>(p.q + (static_cast<int64_t>(st) * p.M + row0 + r) * 64 + 32 * (l >> 5) + 16 * h);
        }
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const int i = i0 + j * T, r = (i >> 7) % TB * 32 + (i & 31);
            if (i < chunks && r < rows) *reinterpret_cast<i32x4*>(panel + i * 16) = v[j];
        }
    }
    for (int i = threadIdx.x; i < nu * TB * 32; i += T) {
        const int k = i / (TB * 32), r = i % (TB * 32);
        if (r < rows) pscale[i] = p.s[(static_cast<int64_t>(k >> 2) * p.M + row0 + r) * 4 + (k & 3)];
    }
}

// The panel made from the rows themselves: 16 lanes a block of a row, F of them in flight.
template <int TB>
__device__ __forceinline__ void f8_quant_panel(const F8Params& p, int row0, int rows, uint8_t* panel, uint8_t* pscale) {
    constexpr int F = 4, G = 16;      // G: groups of 16 lanes
    const int nu = p.kblocks, s = threadIdx.x & 15;
    const int part = p.k.part, part_p = p.k.part_p;
    // the group's items (row, block), G blocks apart
    int r = 0, kb = threadIdx.x >> 4;
    auto wrap = [&]() {
        while (kb >= nu) {
            kb -= nu;
            ++r;
        }
    };
    wrap();
    while (r < rows) {
        uint4 v[F];
        int at[F];       // where the item's values go; -1: no item
        int scale[F];
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const int c = kb * F8_BLOCK + 8 * s, h = c >= part_p, k = c - h * part_p;
            v[j] = make_uint4(0, 0, 0, 0);
            if (r < rows && k < part)
                v[j] = *reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(row0 + r) * p.k.real() + h * part + k);
            // columns 8 s .. of the block: step s / 8, lanes' half s / 4 % 2, operand half s / 2 % 2
            at[j] = r < rows ? ((kb * 2 + (s >> 3)) * TB + (r >> 5)) * 2048 + ((s >> 1) & 1) * 1024 + ((s >> 2) & 1) * 512 +
                                   (r & 31) * 16 + (s & 1) * 8
                             : -1;
            scale[j] = (kb * TB + (r >> 5)) * 32 + (r & 31);
            kb += G;
            wrap();
        }
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const F8Scale sc = f8_scale(f8_top16(f8_top(f8_max2(f8_max2(f8_max2(f8_max2(0, v[j].x), v[j].y), v[j].z), v[j].w))));
            if (at[j] < 0) continue;
            *reinterpret_cast<uint2*>(panel + at[j]) =
                make_uint2(f8_four(lo_f(v[j].x), hi_f(v[j].x), lo_f(v[j].y), hi_f(v[j].y), sc),
                           f8_four(lo_f(v[j].z), hi_f(v[j].z), lo_f(v[j].w), hi_f(v[j].w), sc));
            if (s == 0) pscale[scale[j]] = static_cast<uint8_t>(sc.byte);
        }
    }
}

// ---- Streaming items: a group of rows of one expert x a range of 128-column
// blocks, for which each weight byte is read once; a wave takes 32 columns of a
// block (of each half with F8_STORE_GLU) at a time over the whole summed
// dimension.  Bound by the weights' bytes.
//
// The rows' operands lie in `panel` (LDS, 4 KiB for 32 rows of a block of the
// summed dimension), their scales behind them.  The weights come as one stream
// over a wave's blocks, in units of a block of the summed dimension, all but
// one of R units ahead, the first of them from before the panel is filled:
// nothing drains at a block's end, where the sums go to the epilogue, and
// loads are repeated only at the stretch's own end.  One token's eight experts,
// K = N = 4096: 134 MB in 25 us, 5.4 TB/s.
// R C column blocks of 4 KiB are in flight: 8 (that token 27.5 us with its launch, 28.4 with 12; its gated block 47.3,
// 49.4 with 12 there, 48.8 with 16).
//
// With a quantized output a block's maximum joins four waves' columns over LDS; the block's rows of h1 are loaded
// when the block begins, in front of its weights, so that nothing waits for them at its end.
template <int TB, int EPI, int FP32>
__device__ __forceinline__ void f8_stream_blocks(const F8Params& p, const uint8_t* w, const uint8_t* ws, int row0, int rows,
                                                 int nb0, int nb1, uint8_t* panel, uint32_t (*s_top)[4][F8_GROUP]) {
    constexpr int C = EPI == F8_STORE_GLU ? 2 : 1;   // column blocks of a wave
    constexpr int R = 8 / C;
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), nu = p.kblocks;
    const int total = (nb1 - nb0) * nu;
    const int64_t wblock = static_cast<int64_t>(nu) * 4096;      // bytes of 32 columns
    const int64_t up = EPI == F8_STORE_GLU ? static_cast<int64_t>(p.n.part_p / 32) * wblock : 0;
    const int64_t up_s = EPI == F8_STORE_GLU ? static_cast<int64_t>(p.n.part_p / F8_BLOCK) * p.ws_ld : 0;
    int zero = 0;
    asm volatile("" : "+v"(zero));      // keeps the scales' loads off the scalar unit, whose results come out of order
    const uint8_t* lp = w + (static_cast<int64_t>(nb0) * 4 + wave) * wblock;
    const uint8_t* sp = ws + static_cast<int64_t>(nb0) * p.ws_ld;
    int lk = 0, lf = 0;   // the next unit to load: of its block, and of all
    i32x4 wv[R][C][4];
    int wsv[R][C];
    auto load = [&](i32x4(&v)[C][4], int(&sv)[C]) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                v[c][u] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(lp + c * up + lane * 16 + u * 1024));
            sv[c] = (sp + c * up_s + lk)[zero];
        }
        const bool wrap = ++lk == nu;
        if (++lf < total) {
            lp += 4096 + (wrap ? 3 * wblock : 0);
            sp += wrap ? p.ws_ld : 0;
            lk = wrap ? 0 : lk;
        } else {
            lk = nu - 1;
        }
    };
    f32x16 acc[C][TB];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < TB; ++i) acc[c][i] = f32x16{};
    // in this order: the first unit's wait would otherwise be for all
#pragma unroll
    for (int i = 0; i < R - 1; ++i) {
        load(wv[i], wsv[i]);
        __builtin_amdgcn_sched_barrier(0);
    }
    uint8_t* pscale = panel + F8_PANEL;      // [nu][32 TB]
    __syncthreads();   // the last panel is read
    // What belongs to rows that do not exist stays as it is: a row's products meet no other row's.
    if (p.x) f8_quant_panel<TB>(p, row0, rows, panel, pscale);
    else f8_copy_panel<TB>(p, row0, rows, panel, pscale);
    __syncthreads();
    // a block's rows of h1, loaded when the block begins
    uint2 hg[EPI == F8_STORE_DGLU ? TB : 1][4], hu[EPI == F8_STORE_DGLU ? TB : 1][4];
    int nb = nb0;
    const float e2 = f8_log2e(p.slope);
    auto load_h1 = [&](int b) {
        if constexpr (EPI == F8_STORE_DGLU) {
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                const uint16_t* h = p.h1 + static_cast<int64_t>(row0 + min(i * 32 + (lane & 31), rows - 1)) * 2 * p.n.part;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int c = b * F8_BLOCK + 32 * wave + 8 * q + 4 * (lane >> 5);
                    const bool ok = c < p.n.part;
                    hg[i][q] = ok ? *reinterpret_cast<const uint2*>(h + c) : make_uint2(0, 0);
                    hu[i][q] = ok ? *reinterpret_cast<const uint2*>(h + p.n.part + c) : make_uint2(0, 0);
                }
            }
        }
    };
    load_h1(nb);
    // lane holds row lane & 31 of each 32-row block and, in register 4q + x, column 8q + 4(lane >> 5) + x of the wave's 32
    const int64_t qblock = static_cast<int64_t>(p.M) * 64;
    auto put8 = [&](uint32_t bytes, int r, int c) {     // four 8-bit values from padded column c of row r
        *reinterpret_cast<uint32_t*>(p.q_out + (c >> 6) * qblock + static_cast<int64_t>(row0 + r) * 64 + (c & 63)) = bytes;
    };
    auto put_scale = [&](const F8Scale& s, int r, int kb) {
        p.s_out[(static_cast<int64_t>(kb >> 2) * p.M + row0 + r) * 4 + (kb & 3)] = static_cast<uint8_t>(s.byte);
    };
    // The maxima of a block of 128 columns from those of the waves' 32 each (0 .. PARTS - 1 of them for a row).
    auto block_tops = [&](uint32_t (&top)[TB], int part) {
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            top[i] = max_other_half(f8_top(top[i]));
            if (lane < 32) s_top[part][wave][32 * i + lane] = top[i];
        }
    };
    auto join_tops = [&](uint32_t (&top)[TB], int part) {
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            const int r = 32 * i + (lane & 31);
            top[i] = max(max(s_top[part][0][r], s_top[part][1][r]), max(s_top[part][2][r], s_top[part][3][r]));
        }
    };
    auto epilogue = [&]() {
        const int c0 = nb * F8_BLOCK + 32 * wave;     // padded column
        if constexpr (EPI == F8_STORE) {
            const int h = c0 >= p.n.part_p, k0 = c0 - h * p.n.part_p;
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                const int r = i * 32 + (lane & 31);
                uint16_t* o = p.out + static_cast<int64_t>(row0 + r) * p.n.real() + h * p.n.part;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int k = k0 + 8 * q + 4 * (lane >> 5);
                    if (r < rows && k < p.n.part && nb < nb1)
                        *reinterpret_cast<uint2*>(o + k) = make_uint2(pack2(acc[0][i][4 * q], acc[0][i][4 * q + 1]),
                                                                      pack2(acc[0][i][4 * q + 2], acc[0][i][4 * q + 3]));
                }
            }
        } else {
            constexpr int PARTS = EPI == F8_STORE_DGLU ? 2 : 1;
            uint32_t v[PARTS][TB][8], top[PARTS][TB];
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                const int r = i * 32 + (lane & 31);
#pragma unroll
                for (int h = 0; h < PARTS; ++h) top[h][i] = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int c = c0 + 8 * q + 4 * (lane >> 5);
                    uint2 b[C];
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        b[j] = make_uint2(pack2(acc[j][i][4 * q], acc[j][i][4 * q + 1]),
                                          pack2(acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]));
                    if constexpr (EPI == F8_STORE_GLU) {
                        if (p.out && r < rows && c < p.n.part && nb < nb1) {
                            uint16_t* o = p.out + static_cast<int64_t>(row0 + r) * p.n.real() + c;
                            *reinterpret_cast<uint2*>(o) = b[0];
                            *reinterpret_cast<uint2*>(o + p.n.part) = b[C - 1];
                        }
                        v[0][i][2 * q] = pack2(f8_act(lo_f(b[0].x), lo_f(b[C - 1].x), e2), f8_act(hi_f(b[0].x), hi_f(b[C - 1].x), e2));
                        v[0][i][2 * q + 1] = pack2(f8_act(lo_f(b[0].y), lo_f(b[C - 1].y), e2), f8_act(hi_f(b[0].y), hi_f(b[C - 1].y), e2));
                    } else {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t d = y ? b[0].y : b[0].x, g = y ? hg[i][q].y : hg[i][q].x, u = y ? hu[i][q].y : hu[i][q].x;
                            float g0, u0, g1, u1;
                            f8_act_grad(lo_f(g), lo_f(u), lo_f(d), p.slope, e2, g0, u0);
                            f8_act_grad(hi_f(g), hi_f(u), hi_f(d), p.slope, e2, g1, u1);
                            v[0][i][2 * q + y] = pack2(g0, g1);
                            v[PARTS - 1][i][2 * q + y] = pack2(u0, u1);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < PARTS; ++h)
                        top[h][i] = f8_max2(f8_max2(top[h][i], v[h][i][2 * q]), v[h][i][2 * q + 1]);
                }
            }
            block_barrier();     // the last block's maxima are read
#pragma unroll
            for (int h = 0; h < PARTS; ++h) block_tops(top[h], h);
            block_barrier();
#pragma unroll
            for (int h = 0; h < PARTS; ++h) {
                join_tops(top[h], h);
                const int part_p = p.n.part_p, kb = nb + h * (part_p / F8_BLOCK);
#pragma unroll
                for (int i = 0; i < TB; ++i) {
                    const int r = i * 32 + (lane & 31);
                    const F8Scale sc = f8_scale(top[h][i]);
                    if (r >= rows || nb >= nb1) continue;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t a = v[h][i][2 * q], b = v[h][i][2 * q + 1];
                        put8(f8_four(lo_f(a), hi_f(a), lo_f(b), hi_f(b), sc), r, h * part_p + c0 + 8 * q + 4 * (lane >> 5));
                    }
                    if (wave == 0 && lane < 32) put_scale(sc, r, kb);
                }
            }
        }
    };
    int k = 0;
    for (int f = 0; f < total; f += R) {
        // the last round's units past the end multiply what was loaded last and are not stored
        static_for<R>([&](auto i_tag) {
            constexpr int at = decltype(i_tag)::value;
            load(wv[(at + R - 1) % R], wsv[(at + R - 1) % R]);
            const uint8_t* op = panel + k * (TB * 4096) + lane * 16;
            int ts[TB];
#pragma unroll
            for (int i = 0; i < TB; ++i) ts[i] = pscale[(k * TB + i) * 32 + (lane & 31)];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < TB; ++i) {
                    const uint8_t* o = op + (u * TB + i) * 2048;
                    const i32x8 t = f8_join(*reinterpret_cast<const i32x4*>(o), *reinterpret_cast<const i32x4*>(o + 1024));
                    if constexpr (FP32 == 0) {
#pragma unroll
                        for (int c = 0; c < C; ++c)
                            acc[c][i] = f8_mma(f8_join(wv[at][c][2 * u], wv[at][c][2 * u + 1]), t, acc[c][i], wsv[at][c], ts[i]);
                    } else {
                        static_for<4>([&](auto s_tag) {
                            constexpr int s = decltype(s_tag)::value;
                            const f8_bf16x8 tb = f8_eight<s>(t, f8_row_factor(ts[i]));
#pragma unroll
                            for (int c = 0; c < C; ++c)
                                acc[c][i] = f8_mma_bf16(f8_eight<s>(f8_join(wv[at][c][2 * u], wv[at][c][2 * u + 1]),
                                                                    f8_weight_factor(static_cast<uint32_t>(wsv[at][c]))),
                                                        tb, acc[c][i]);
                        });
                    }
                }
            if (++k == nu) {
                k = 0;
                epilogue();
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < TB; ++i) acc[c][i] = f32x16{};
                ++nb;
                load_h1(min(nb, nb1 - 1));
            }
        });
    }
}

// The list of all (row group, 128-column block) pairs, in equal stretches to the workgroups.  s_off, s_pre: [E + 1].
//
// Next to tiles, experts that fit one item are streamed, whole.  (A large expert's last rows as a partial tile cost
// less than the weights read once more for them: 128 experts of 320 rows, K 768, N 2048: 129 us, 153 us with remainders of
// up to 96 rows streamed; 32 of 300 rows, the gated block's gradient: 121 us, 156.)
template <int EPI, int FP32>
__device__ __forceinline__ void f8_stream_list(const F8Params& p, int* s_off, int* s_pre, uint8_t* panel,
                                               uint32_t (*s_top)[4][F8_GROUP]) {
    const int nblocks = EPI == F8_STORE_GLU ? p.n.part_p / F8_BLOCK : p.n.blocks();
    prefix_experts(p.offsets, p.E, p.M, s_off, s_pre,
                   [&](int m) { return p.tile && m > p.group ? 0 : (m + p.group - 1) / p.group * nblocks; });
    const int64_t total = uni(s_pre[p.E]);
    int at = static_cast<int>(total * blockIdx.x / gridDim.x);
    const int end = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
    while (at < end) {   // one row group's part of the stretch
        const int e = uni(find_expert_wave(s_pre, p.E, at));
        const int local = at - uni(s_pre[e]), grp = local / nblocks, nb0 = local - grp * nblocks;
        const int nb1 = min(nblocks, nb0 + end - at);
        const int lo = uni(s_off[e]), hi = uni(s_off[e + 1]);
        const int row0 = lo + grp * p.group;
        const int rows = min(p.group, hi - row0);
        const uint8_t* w = p.w + static_cast<int64_t>(e) * p.w_stride;
        const uint8_t* ws = p.ws + static_cast<int64_t>(e) * p.ws_stride;
        const int tb = (rows + 31) / 32;
        if (tb == 1) f8_stream_blocks<1, EPI, FP32>(p, w, ws, row0, rows, nb0, nb1, panel, s_top);
        else f8_stream_blocks<2, EPI, FP32>(p, w, ws, row0, rows, nb0, nb1, panel, s_top);
        at += nb1 - nb0;
    }
}

template <int EPI, int FP32>
__global__ __launch_bounds__(256, 1) void f8_stream_kernel(const F8Params p) {
    __shared__ __attribute__((aligned(1024))) uint8_t s_ring[F8_RING];
    __shared__ uint32_t s_top[2][4][F8_GROUP];
    __shared__ int s_off[GG_KMAX_EXPERTS + 1];
    __shared__ int s_pre[GG_KMAX_EXPERTS + 1];
    f8_stream_list<EPI, FP32>(p, s_off, s_pre, s_ring, s_top);
}

// A value kept in an accumulation register, and back.
__device__ __forceinline__ float acc_wr(uint32_t v) {
    float a;
    asm volatile("v_accvgpr_write_b32 %0, %1" : "=a"(a) : "v"(v));
    return a;
}
__device__ __forceinline__ uint32_t acc_rd_u(float a) { return __builtin_bit_cast(uint32_t, acc_rd(a)); }

constexpr int F8_STAGE = 64;
constexpr int F8_STG_BYTES = 32 * 128;   // per wave: 32 rows x 64 columns of bf16

// ---- Tiles: 64 BR rows x 64 BC packed columns by four waves, each 32 BR x
// 32 BC, as BR x BC accumulators of 32 x 32: 256 x 256 (the accumulators fill half the registers), 128 x 256 and, for
// F8_STORE, 128 x 128.  With F8_STORE_GLU a wave's columns are half gate, half
// the same columns of up, so that A is made where the sums are; two waves join
// their maxima of a block of A.  With F8_STORE_DGLU a wave's columns are a block of dA.
//
// Rows, their scales and weights stream into an LDS ring of 64-column stages by
// LDS-DMA: the rows, 16-byte chunk c of row r at c ^ ((r >> 2) & 3), the weights
// as they lie in the packed layout (fragment reads of both are free of bank
// conflicts), and for each row the dword with the scale of the stage's block.
// The copies of a workgroup's tiles are one sequence, a ring ahead of the
// products: a tile's first stages land during the last tile's last stages and
// its epilogue (32768 rows, K 1536, N 2048: 157 us with a ramp for
// each tile, and some spilled registers, 111 us so).
// A stage is BR x BC matrix instructions a wave.  After the first BC of them
// the next stage has landed and every wave holds its fragments of this one,
// whose slot is refilled from there on; behind each of the other instructions
// come one fragment's reads of the next stage and one copy.  The epilogue goes
// through a small staging area of its own, and the waits of the next tile's
// first stages leave its stores outstanding: memory operations complete in
// order.
//
// 262144 rows, K = N = 4096: 3.3 ms, 2.7 PFLOP/s (a library's product with one scale a tensor 2.8).  The matrix pipe is
// busy 72% of the cycles and the clock at 1.5 to 1.8 GHz: the chip's power is the bound.  K 768, 131072 rows, N 2048: 265 us,
// 1.6 PFLOP/s: besides its 12 stages a tile waits about 6 us for its 128 KiB of stores, 3 us of them for the first
// one, as the loads behind them count only when they are done.  Two workgroups of 128 x 256 on a CU hide that wait but
// read half as much again (the first case 20% slower, the second equal).
template <int BR, int BC, int EPI, int FP32>
__global__ __launch_bounds__(256, 1) void f8_tile_kernel(const F8Params p) {
    constexpr int TR = 64 * BR, TC = 64 * BC;               // rows and packed columns of a tile
    constexpr int OC = EPI == F8_STORE_GLU ? TC / 2 : TC;   // columns of what it makes
    static_assert(EPI == F8_STORE || BC == 4, "a quantized block's columns lie in one tile");
    constexpr int W_AT = TR * F8_STAGE, S_AT = W_AT + TC * F8_STAGE;
    constexpr int SLOT_BYTES = S_AT + TR * 4, SLOTS = BR == 4 ? 4 : (BC == 4 ? 4 : 8);
    static_assert(SLOTS * SLOT_BYTES <= F8_RING, "the ring");
    constexpr int P = BR + BC + 1;                          // copies a wave issues for a stage
    constexpr int READS_A_STEP = BR == 4 ? 1 : 2;           // fragments read behind a matrix instruction
    constexpr int WS = EPI == F8_STORE_GLU ? 2 : 1;         // blocks of weights that a wave's columns lie in
    __shared__ __attribute__((aligned(1024))) uint8_t s_ring[F8_RING];
    __shared__ __attribute__((aligned(16))) uint8_t s_stg[4 * F8_STG_BYTES];
    __shared__ uint32_t s_row_top[EPI == F8_STORE_GLU ? 4 * 32 * BR : 1];
    __shared__ int s_off[GG_KMAX_EXPERTS + 1];
    __shared__ int s_pre[GG_KMAX_EXPERTS + 1];
    const int nsteps = p.kblocks * 2, nstages = nsteps;
    const int part_p = p.n.part_p, width = EPI == F8_STORE_GLU ? part_p : p.n.padded();
    const int tiles_n = (width + OC - 1) / OC;
    // The 32 tiles that an XCD works on at a time are about as many row as column tiles, whose operands its L2 holds.
    const int band = max(4, 32 / tiles_n);
    const auto tiles_of = [&](int m) { return m <= p.group ? 0 : (m - 1) / TR + 1; };     // row tiles of an expert
    prefix_experts(p.offsets, p.E, p.M, s_off, s_pre, [&](int m) { return tiles_of(m) * tiles_n; });
    const int n_tiles = uni(s_pre[p.E]);
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int wr = wave >> 1, wc = wave & 1;      // the wave's rows and columns
    // consecutive tiles to the workgroups of one XCD, which share an L2
    const int G = gridDim.x, b = blockIdx.x;
    const int slot = (G % 8 == 0) ? (b & 7) * (G >> 3) + (b >> 3) : b;
    const uint32_t ring = lds_addr(s_ring);

    // A tile: its expert's rows [row0, row0 + rows), its columns from col0 on, and the scales of this wave's columns
    // (F8_STORE_GLU: of gate and up).
    struct Tile {
        int row0, rows, col0;
        const uint8_t* ws[WS];
    } next;
    // The copies' cursor: what a stage's copies of `next` read, moved on a stage at a time.
    const uint8_t *t_ptr = nullptr, *w_ptr = nullptr, *s_ptr = nullptr;   // first row, its expert's matrix, first row's scales
    uint32_t t_voff[BR], s_voff;       // this lane's chunks of rows 16 BR wave + 16 i .., its scale
    uint32_t w_voff[BC / 2];           // its part of each 32-column block that this wave copies
    uint32_t wd_first[WS];             // the weights' scales of the first four blocks
    int c_at = 0;                      // the stage
    const int64_t t_block = static_cast<int64_t>(p.M) * F8_STAGE;   // bytes of 64 columns of all rows
    const int64_t s_block = static_cast<int64_t>(p.M) * 4;          // and of four blocks' scales
    auto setup = [&](int t) {
        const int e = uni(find_expert_wave(s_pre, p.E, t));
        const int local = t - uni(s_pre[e]);
        const int lo = uni(s_off[e]), m = uni(s_off[e + 1]) - lo, tiles_m = tiles_of(m);
        // groups of `band` row tiles, columns by columns
        const int g = local / (band * tiles_n), r = local - g * band * tiles_n, high = min(band, tiles_m - g * band);
        const int tm = g * band + r % high, tn = r / high;
        next.row0 = lo + tm * TR;
        next.rows = min(TR, m - tm * TR);
        next.col0 = tn * OC;
        t_ptr = p.q + static_cast<int64_t>(next.row0) * F8_STAGE;
        s_ptr = p.s + static_cast<int64_t>(next.row0) * 4;
        w_ptr = p.w + static_cast<int64_t>(e) * p.w_stride;
        const uint8_t* ws = p.ws + static_cast<int64_t>(e) * p.ws_stride;
        const int rb = next.col0 / F8_BLOCK + (EPI != F8_STORE_GLU && BC == 4 ? wc : 0);
        next.ws[0] = ws + static_cast<int64_t>(min(rb, p.n.blocks() - 1)) * p.ws_ld;
        if constexpr (WS == 2) next.ws[1] = next.ws[0] + static_cast<int64_t>(part_p / F8_BLOCK) * p.ws_ld;
#pragma unroll
        for (int c = 0; c < WS; ++c) wd_first[c] = scalar_load(next.ws[c]);
#pragma unroll
        for (int i = 0; i < BR; ++i) {
            const int r = 16 * BR * wave + 16 * i + (lane >> 2);
            const int c = (lane & 3) ^ ((r >> 2) & 3);
            t_voff[i] = static_cast<uint32_t>(min(r, next.rows - 1)) * F8_STAGE + 16 * c;
        }
        s_voff = static_cast<uint32_t>(min((64 * wave + lane) & (TR - 1), next.rows - 1)) * 4;
#pragma unroll
        for (int i = 0; i < BC / 2; ++i) {
            const int at = wave * (BC / 2) + i;           // the block's place in the tile
            int wb;
            if constexpr (EPI == F8_STORE_GLU)            // each wave column: two gate blocks, then two of up
                wb = ((at & 3) >> 1) * (part_p / 32) + next.col0 / 32 + 2 * (at >> 2) + (at & 1);
            else
                wb = min(next.col0 / 32 + at, width / 32 - 1);
            w_voff[i] = static_cast<uint32_t>(wb) * static_cast<uint32_t>(nstages * 2048) + lane * 16;    // below 2^31
        }
        c_at = 0;
    };
    // One of the P copies of the cursor's stage that this wave issues, to the slot at LDS offset `slot_at`.
    auto piece = [&](uint32_t slot_at, auto i_tag) {
        constexpr int i = decltype(i_tag)::value;
        const uint32_t dst = ring + slot_at;
        if constexpr (i < BR) {
            dma16(t_ptr, t_voff[i], dst + (16 * BR * wave + 16 * i) * F8_STAGE);
        } else if constexpr (i < BR + BC) {
            constexpr int j = (i - BR) / 2, h = (i - BR) % 2;
            dma16_at<1024 * h>(w_ptr, w_voff[j], dst + W_AT + (wave * (BC / 2) + j) * 2048);
        } else {
            dma4(s_ptr, s_voff, dst + S_AT + ((64 * wave) & (TR - 1)) * 4);
        }
    };
    // A tile has two stages more than the ring at least (of a shorter sum, the last ones are copied but not multiplied),
    // so that the cursor, a ring ahead, is never more than a tile ahead.
    const int nst = max(nstages, SLOTS + 2);
    int t = slot;
    // Behind a stage's copies: the cursor moves to the next stage, of the next tile after a tile's last (of the same
    // one again where there is none: those copies are not used).
    auto advance = [&]() {
        ++c_at;
        if (c_at < nstages) {
            t_ptr += t_block;
            w_ptr += 2048;
            if ((c_at & 7) == 0) s_ptr += s_block;
        }
        if (c_at == nst) setup(t + G < n_tiles ? t + G : t);
    };

    f32x16 acc[BR][BC];    // [row block][column block]
    constexpr int SETS = FP32 ? 1 : 2;      // of fragments as they are read
    i32x8 tf[SETS][BR], wf[SETS][BC];
    f8_bf16x8 tb[2][4], wb[BC][4];          // FP32: as bf16, rows of two row blocks
    int ts[BR], ts_next[BR], wsc[WS];       // scales of the block that is multiplied, and of the next
    uint32_t wd[WS], wd_next[WS];           // the weights' scales, four blocks in a dword
    // a lane's first 16 bytes of a fragment in a slot; its second are 16 bytes off in the swizzled rows
    const uint32_t t_at = (32 * BR * wr + (lane & 31)) * F8_STAGE + 16 * ((2 * (lane >> 5)) ^ ((lane >> 2) & 3));
    const uint32_t w_at = W_AT + BC * wc * 2048 + lane * 16, s_at = S_AT + (32 * BR * wr + (lane & 31)) * 4;
    // fragment i of the slot at sl, of the parity u
    auto read_t = [&](uint32_t sl, auto i_tag, auto u_tag) {
        constexpr int u = decltype(u_tag)::value % SETS, i = decltype(i_tag)::value;
        tf[u][i] = f8_join(*reinterpret_cast<const i32x4*>(s_ring + (sl + t_at) + i * 32 * F8_STAGE),
                           *reinterpret_cast<const i32x4*>(s_ring + (sl + (t_at ^ 16)) + i * 32 * F8_STAGE));
    };
    auto read_w = [&](uint32_t sl, auto j_tag, auto u_tag) {
        constexpr int u = decltype(u_tag)::value % SETS, j = decltype(j_tag)::value;
        const uint8_t* f = s_ring + (sl + w_at) + j * 2048;
        wf[u][j] = f8_join(*reinterpret_cast<const i32x4*>(f), *reinterpret_cast<const i32x4*>(f + 1024));
    };
    // the rows' scales of the stage's block kb, with the first of a block's two stages
    auto read_s = [&](uint32_t sl, int kb) {
        const uint8_t* sc = s_ring + (sl + s_at + (kb & 3));
#pragma unroll
        for (int i = 0; i < BR; ++i) ts_next[i] = sc[i * 128];
    };
    // Read f of a stage's BR + BC, in the order in which the next stage needs them.
    auto read = [&](uint32_t sl, auto f_tag, auto u_tag) {
        constexpr int f = decltype(f_tag)::value;
        if constexpr (f == 0) read_t(sl, GrpTag<0>{}, u_tag);
        else if constexpr (f <= BC) read_w(sl, GrpTag<f - 1>{}, u_tag);
        else read_t(sl, GrpTag<f - BC>{}, u_tag);
    };
    // matrix instruction m of a stage, rows first; the tile's first stage starts its sums from zero
    auto mma = [&](auto u_tag, auto m_tag, auto first_tag) {
        constexpr int u = decltype(u_tag)::value % SETS, i = decltype(m_tag)::value / BC, j = decltype(m_tag)::value % BC;
        const int s = wsc[WS == 2 && j >= BC / 2];
        if constexpr (decltype(first_tag)::value != 0)
            acc[i][j] = f8_mma(wf[u][j], tf[u][i], f32x16{}, s, ts[i]);
        else
            acc[i][j] = f8_mma(wf[u][j], tf[u][i], acc[i][j], s, ts[i]);
        asm volatile("" : "+a"(acc[i][j]));     // in its place: the compiler sinks matrix instructions past branches
    };
    // FP32: eights s of the weights of block j as bf16
    auto weights_bf16 = [&](auto j_tag, auto s_tag, uint32_t byte) {
        constexpr int j = decltype(j_tag)::value, s = decltype(s_tag)::value;
        wb[j][s] = f8_eight<s>(wf[0][j], f8_weight_factor(byte));
        asm volatile("" : "+v"(wb[j][s]));      // in its place, as the matrix instructions
    };
    auto fence = [&]() { __builtin_amdgcn_sched_barrier(0); };
    // Waits until the next stage has landed: the copies of the ring's other stages, and `behind` stores among them, may
    // be outstanding.
    constexpr int AHEAD = P * (SLOTS - 2);
    constexpr int S1 = EPI == F8_STORE ? 2 * BR * BC : (EPI == F8_STORE_GLU ? 2 * BR : 8 * BR);   // of a full tile
    constexpr int S2 = S1 + (EPI == F8_STORE_GLU ? 8 * BR : 0);                                   // with H1
    constexpr int MOST = 63;
    auto wait_ahead = [&](int behind) {
        if (behind == 0) wait_vmcnt<AHEAD>();
        else if (S2 == S1 || behind == S1) wait_vmcnt<(AHEAD + S1 < MOST ? AHEAD + S1 : MOST)>();
        else wait_vmcnt<(AHEAD + S2 < MOST ? AHEAD + S2 : MOST)>();
    };
    // Stage st of the tile, of the parity u, in the slot at cur.  behind: the stores issued behind the copies of the
    // ring's other stages.  After the tile's last stage the next fragments belong to another tile; they are read again
    // after the epilogue.
    uint32_t cur = 0;
    const uint8_t* cur_ws[WS];
    // The stages and what they call are inlined by force: a call would put the accumulators into memory.
    //
    // the scales of block k, where it begins
    auto roll_scales = [&](int k) {
#pragma unroll
        for (int i = 0; i < BR; ++i) ts[i] = ts_next[i];
        if ((k & 3) == 0) {
#pragma unroll
            for (int c = 0; c < WS; ++c) {
                wd[c] = wd_next[c];
                wd_next[c] = scalar_load(cur_ws[c] + min(k + 4, p.ws_ld - 4));
            }
        }
#pragma unroll
        for (int c = 0; c < WS; ++c) wsc[c] = static_cast<int>(wd[c] >> (8 * (k & 3)));
    };
    // The stage with fp32 sums: four bf16 instructions for each scaled one.  Of its BR x 4 slots, slot (i, s) multiplies
    // eights s of row block i by those of all columns.  Behind a slot's instructions eights of the next row block become
    // bf16, and behind the last row block's those of the next stage's weights and first row block, in the registers that
    // are read for the last time there.  So fragments are read into one set of registers, and a conversion waits for
    // neither a read nor an instruction: two of 8 cycles go with an instruction of 32 (up to four in a loop of nothing
    // else take no time; where the compiler had moved them to their use, the tiles took 10% more).
    //
    // 65536 rows, H 4096, F 2048, H1 and A: 1.89 ms (matrix pipe 69% busy at 1.6 GHz: the chip's power), 1.01 with scaled sums.
    auto stage_fp32 = [&](int st, int behind, auto u_tag, auto first_tag) __attribute__((always_inline)) {
        constexpr int u = decltype(u_tag)::value;
        if constexpr (u == 0) roll_scales(st >> 1);
        constexpr int Q = 4 * BR, SYNC = BR == 4 ? 3 : 0, REST = Q - 1 - SYNC;
        uint32_t refill = 0;
        uint32_t wnext[WS];     // the weights' scales of the next stage
        static_for<Q>([&](auto q_tag) {
            constexpr int q = decltype(q_tag)::value, i = q / 4, s = q % 4;
            if constexpr (q == 4 * (BR - 1)) {
#pragma unroll
                for (int c = 0; c < WS; ++c) {
                    const int k = (st + 1) >> 1;
                    wnext[c] = u == 0 ? static_cast<uint32_t>(wsc[c]) : ((k & 3) == 0 ? wd_next[c] : wd[c]) >> (8 * (k & 3));
                    wnext[c] &= 255;
                }
            }
            static_for<BC>([&](auto j_tag) {
                constexpr int j = decltype(j_tag)::value;
                if constexpr (decltype(first_tag)::value != 0 && s == 0)
                    acc[i][j] = f8_mma_bf16(wb[j][s], tb[i % 2][s], f32x16{});
                else
                    acc[i][j] = f8_mma_bf16(wb[j][s], tb[i % 2][s], acc[i][j]);
                asm volatile("" : "+a"(acc[i][j]));
                if constexpr (i < BR - 1) {
                    static_for<4 / BC>([&](auto y) {
                        f8_pair<s, j * (4 / BC) + decltype(y)::value>(tb[(i + 1) % 2][s], tf[0][i + 1], f8_row_factor(ts[i + 1]));
                    });
                    if constexpr (j == BC - 1) asm volatile("" : "+v"(tb[(i + 1) % 2][s]));
                } else {
                    weights_bf16(j_tag, GrpTag<s>{}, wnext[WS == 2 && j >= BC / 2]);
                    static_for<4 / BC>([&](auto y) {
                        f8_pair<s, j * (4 / BC) + decltype(y)::value>(tb[0][s], tf[0][0], f8_row_factor(u == 0 ? ts[0] : ts_next[0]));
                    });
                    if constexpr (j == BC - 1) asm volatile("" : "+v"(tb[0][s]));
                }
                fence();
            });
            if constexpr (q == SYNC) {
                // stage st + 1 has landed, and every wave holds its fragments of stage st, as in stage()
                wait_ahead(behind);
                block_barrier();
                refill = cur;
                cur = cur + SLOT_BYTES == SLOTS * SLOT_BYTES ? 0 : cur + SLOT_BYTES;
            } else if constexpr (q > SYNC) {
                constexpr int m = q - SYNC - 1;
                if constexpr (u == 1 && m == 0) read_s(cur, (st + 1) >> 1);
                // the first row block and the weights before the last row block's slots; row block i > 0 when it has become bf16
                constexpr int BEFORE = BR == 4 ? 5 : 2, EACH = (BC + 1 + BEFORE - 1) / BEFORE;
                constexpr int f0 = m * EACH, f1 = f0 + EACH;
                static_for<(f1 < BC + 1 ? f1 : BC + 1) - (f0 < BC + 1 ? f0 : BC + 1)>(
                    [&](auto f) { read(cur, GrpTag<f0 + decltype(f)::value>{}, GrpTag<0>{}); });
                static_for<BR - 1>([&](auto r_tag) {
                    constexpr int r = decltype(r_tag)::value + 1, after = BR == 4 && r == 1 ? 9 : (BR == 4 && r == 2 ? 10 : 4 * r);
                    if constexpr (q == after) read_t(cur, GrpTag<r>{}, GrpTag<0>{});
                });
                constexpr int a = m * P / REST, z = (m + 1) * P / REST;
                static_for<z - a>([&](auto j) { piece(refill, GrpTag<a + decltype(j)::value>{}); });
                fence();
            }
        });
        advance();
    };
    auto stage_scaled = [&](int st, int behind, auto u_tag, auto first_tag) __attribute__((always_inline)) {
        constexpr int u = decltype(u_tag)::value;
        if constexpr (u == 0) roll_scales(st >> 1);
        static_for<BC>([&](auto m) { mma(u_tag, m, first_tag); });
        fence();
        // stage st + 1 has landed, and every wave holds its fragments of stage st, whose slot is refilled from here on
        wait_ahead(behind);
        block_barrier();
        const uint32_t refill = cur;
        cur = cur + SLOT_BYTES == SLOTS * SLOT_BYTES ? 0 : cur + SLOT_BYTES;
        // behind each of the other matrix instructions a fragment's reads and a copy, so that neither holds them up
        constexpr int REST = BR * BC - BC, FR = BR + BC;
        static_for<REST>([&](auto m_tag) {
            constexpr int m = decltype(m_tag)::value;
            mma(u_tag, GrpTag<m + BC>{}, first_tag);
            if constexpr (u == 1 && m == 0) read_s(cur, (st + 1) >> 1);
            constexpr int f0 = m * READS_A_STEP, f1 = (m + 1) * READS_A_STEP;
            static_for<(f1 < FR ? f1 : FR) - (f0 < FR ? f0 : FR)>(
                [&](auto f) { read(cur, GrpTag<f0 + decltype(f)::value>{}, GrpTag<u ^ 1>{}); });
            constexpr int a = m * P / REST, z = (m + 1) * P / REST;
            static_for<z - a>([&](auto j) { piece(refill, GrpTag<a + decltype(j)::value>{}); });
            fence();
        });
        advance();
    };
    auto stage = [&](int st, int behind, auto u_tag, auto first_tag) __attribute__((always_inline)) {
        if constexpr (FP32) stage_fp32(st, behind, u_tag, first_tag);
        else stage_scaled(st, behind, u_tag, first_tag);
    };

    // a stage without products
    auto idle = [&](int behind) {
        wait_ahead(behind);
        block_barrier();
        const uint32_t refill = cur;
        cur = cur + SLOT_BYTES == SLOTS * SLOT_BYTES ? 0 : cur + SLOT_BYTES;
        static_for<P>([&](auto j) { piece(refill, j); });
        advance();
    };

    int stores = 0;
    Tile tile;
    if (t < n_tiles) {
        setup(t);
        tile = next;
#pragma unroll
        for (int c = 0; c < WS; ++c) wd_next[c] = wd_first[c];
#pragma unroll 1
        for (uint32_t at = 0; at < SLOTS * SLOT_BYTES; at += SLOT_BYTES) {
            static_for<P>([&](auto j) { piece(at, j); });
            advance();
        }
        wait_vmcnt<P*(SLOTS - 1)>();
        block_barrier();
    }
    while (t < n_tiles) {
#pragma unroll
        for (int c = 0; c < WS; ++c) cur_ws[c] = tile.ws[c];
        read_s(cur, 0);
        static_for<BR + BC>([&](auto f) { read(cur, f, GrpTag<0>{}); });
        if constexpr (FP32)
            static_for<4>([&](auto s_tag) {
                static_for<BC>([&](auto j_tag) {
                    weights_bf16(j_tag, s_tag, wd_next[WS == 2 && decltype(j_tag)::value >= BC / 2] & 255);
                });
                tb[0][decltype(s_tag)::value] = f8_eight<decltype(s_tag)::value>(tf[0][0], f8_row_factor(ts_next[0]));
            });
        stage(0, stores, GrpTag<0>{}, GrpTag<1>{});     // an even number of stages, at least two
        stage(1, stores, GrpTag<1>{}, GrpTag<0>{});
#pragma unroll 1
        for (int st = 2; st < nstages; st += 2) {
            stage(st, st < SLOTS - 1 ? stores : 0, GrpTag<0>{}, GrpTag<0>{});
            stage(st + 1, st + 1 < SLOTS - 1 ? stores : 0, GrpTag<1>{}, GrpTag<0>{});
        }
#pragma unroll 1
        for (int st = nstages; st < nst; ++st) idle(st < SLOTS - 1 ? stores : 0);
        const int prow0 = tile.row0, prows = tile.rows, pcol0 = tile.col0;
        mfma_drain();
        int opaque = 0;
        asm volatile("" : "+s"(opaque));
        const int ln = lane + opaque;
        uint16_t* stg = reinterpret_cast<uint16_t*>(s_stg + wave * F8_STG_BYTES) + opaque;
        // Blocks of 32 rows x 64 bf16 columns go through the staging area, [32 rows][64 columns] with 16-byte chunk c
        // of row r at c ^ (r & 7); lane's part of the sums: row ln & 31, columns 8 c + 4 (ln >> 5) .. + 3.
        auto put = [&](const uint2 (&v)[8]) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int rr = ln & 31;
                *reinterpret_cast<uint2*>(stg + rr * 64 + ((c ^ (rr & 7)) << 3) + 4 * (ln >> 5)) = v[c];
            }
        };
        auto take = [&](uint2 (&v)[8]) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int rr = ln & 31;
                v[c] = *reinterpret_cast<const uint2*>(stg + rr * 64 + ((c ^ (rr & 7)) << 3) + 4 * (ln >> 5));
            }
        };
        // the same block by rows: lane has row 8 k + (ln >> 3), 16-byte chunk (ln & 7) ^ (ln >> 3)
        auto rows_of = [&](uint4 (&o)[4]) {
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = *reinterpret_cast<const uint4*>(stg + (8 * k + (ln >> 3)) * 64 + (ln & 7) * 8);
        };
        const int chunk = 8 * ((ln & 7) ^ (ln >> 3));
        // the bf16 sums of block (i, column blocks 2 jh and 2 jh + 1)
        auto sums = [&](auto i_tag, auto jh_tag, uint2 (&v)[8]) {
            constexpr int i = decltype(i_tag)::value, jh = decltype(jh_tag)::value;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const f32x16& a = acc[i][2 * jh + (c >> 2)];
                const int q = c & 3;
                v[c] = make_uint2(pack2(acc_rd(a[4 * q]), acc_rd(a[4 * q + 1])), pack2(acc_rd(a[4 * q + 2]), acc_rd(a[4 * q + 3])));
            }
        };
        // a block's rows to columns col .. of `to` (row stride ld), of which those below `cols` exist
        auto store = [&](const uint4 (&o)[4], uint16_t* to, int64_t ld, int i, int cols, auto full_tag) {
            const int gr = 32 * BR * wr + 32 * i + (ln >> 3);
            uint16_t* at = to + static_cast<int64_t>(prow0 + gr) * ld + chunk;
            if constexpr (decltype(full_tag)::value != 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) st16_nt(at + static_cast<int64_t>(8 * k) * ld, o[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (gr + 8 * k < prows && chunk < cols) st16_nt(at + static_cast<int64_t>(8 * k) * ld, o[k]);
            }
        };
        // 32 rows x 64 8-bit columns, of which lane has row ln & 31 and the dwords d[c] of columns 8 c + 4 (ln >> 5),
        // through half of the staging area ([32 rows][64 bytes], chunk c of row r at c ^ ((r >> 2) & 3)) to padded column col
        const int64_t qblock = static_cast<int64_t>(p.M) * 64;
        auto store8 = [&](const uint32_t (&d)[8], int half, int i, int col, auto full_tag) {
            uint8_t* st8 = reinterpret_cast<uint8_t*>(stg) + half * 2048;
            const int rr = ln & 31;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint32_t*>(st8 + rr * 64 + (((c >> 1) ^ ((rr >> 2) & 3)) << 4) + 8 * (c & 1) + 4 * (ln >> 5)) = d[c];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = 16 * k + (ln >> 2), gr = 32 * BR * wr + 32 * i + r;
                const uint4 v = *reinterpret_cast<const uint4*>(st8 + r * 64 + (((ln & 3) ^ ((r >> 2) & 3)) << 4));
                if (decltype(full_tag)::value != 0 || gr < prows)
                    *reinterpret_cast<uint4*>(p.q_out + (col >> 6) * qblock + static_cast<int64_t>(prow0 + gr) * 64 + 16 * (ln & 3)) = v;
            }
        };
        auto store_scale = [&](const F8Scale& sc, int i, int kb, auto full_tag) {     // lanes below 32
            const int gr = 32 * BR * wr + 32 * i + ln;
            if (ln < 32 && (decltype(full_tag)::value != 0 || gr < prows))
                p.s_out[(static_cast<int64_t>(kb >> 2) * p.M + prow0 + gr) * 4 + (kb & 3)] = static_cast<uint8_t>(sc.byte);
        };
        const bool all_rows = prows == TR;
        const float e2 = f8_log2e(p.slope);
        // All stores of a wave are issued where the tile is full; a store whose lanes all lie outside may be
        // skipped, so a partial tile counts as none.
        bool full = all_rows;
        if constexpr (EPI == F8_STORE) full &= (p.n.parts == 1 || p.n.part == part_p) && pcol0 + TC <= p.n.real();
        if constexpr (EPI == F8_STORE_GLU) full &= pcol0 + OC <= p.n.part;
        if constexpr (EPI == F8_STORE_DGLU) full &= pcol0 + OC <= part_p;
        stores = full ? (EPI == F8_STORE_GLU && p.out ? S2 : S1) : 0;
        auto epilogue = [&](auto full_tag) {
            if constexpr (EPI == F8_STORE) {
                const int gc0 = pcol0 + 32 * BC * wc;
                uint2 vals[8];
                sums(GrpTag<0>{}, GrpTag<0>{}, vals);
                put(vals);
                static_for<BR * BC / 2>([&](auto b_tag) {
                    constexpr int blk = decltype(b_tag)::value, i = blk % BR, jh = blk / BR, nx = blk + 1;
                    if constexpr (nx < BR * BC / 2) sums(GrpTag<nx % BR>{}, GrpTag<nx / BR>{}, vals);
                    uint4 out[4];
                    rows_of(out);
                    if constexpr (nx < BR * BC / 2) put(vals);
                    const int c = gc0 + 64 * jh, h = p.n.parts == 2 && c >= part_p, k = c - h * part_p;
                    store(out, p.out + h * p.n.part + k, p.n.real(), i, p.n.part - k, full_tag);
                });
            } else if constexpr (EPI == F8_STORE_GLU) {
                const int k0 = pcol0 + 64 * wc;          // the wave's 64 columns of gate, up and A
                uint32_t av[BR][16], top[BR];
                static_for<BR>([&](auto i_tag) {
                    constexpr int i = decltype(i_tag)::value;
                    uint2 g[8], u[8];
                    sums(i_tag, GrpTag<0>{}, g);
                    sums(i_tag, GrpTag<1>{}, u);
                    top[i] = 0;
                    auto act = [&](int c0) {
#pragma unroll
                        for (int c = c0; c < c0 + 4; ++c) {
                            av[i][2 * c] = pack2(f8_act(lo_f(g[c].x), lo_f(u[c].x), e2), f8_act(hi_f(g[c].x), hi_f(u[c].x), e2));
                            av[i][2 * c + 1] = pack2(f8_act(lo_f(g[c].y), lo_f(u[c].y), e2), f8_act(hi_f(g[c].y), hi_f(u[c].y), e2));
                            top[i] = f8_max2(f8_max2(top[i], av[i][2 * c]), av[i][2 * c + 1]);
                        }
                    };
                    // the arithmetic covers the staging area's round trips
                    uint4 o[4];
                    if (p.out) {
                        put(g);
                        rows_of(o);
                        put(u);
                    }
                    fence();
                    act(0);
                    fence();
                    if (p.out) {
                        store(o, p.out + k0, p.n.real(), i, p.n.part - k0, full_tag);
                        rows_of(o);
                    }
                    fence();
                    act(4);
                    top[i] = max_other_half(f8_top(top[i]));
                    if (ln < 32) s_row_top[wave * 32 * BR + 32 * i + ln] = top[i];
                    fence();
                    if (p.out) store(o, p.out + p.n.part + k0, p.n.real(), i, p.n.part - k0, full_tag);
                });
                block_barrier();
#pragma unroll
                for (int i = 0; i < BR; ++i) {
                    const F8Scale sc = f8_scale(max(top[i], s_row_top[(wave ^ 1) * 32 * BR + 32 * i + (ln & 31)]));
                    uint32_t d[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        d[c] = f8_four(lo_f(av[i][2 * c]), hi_f(av[i][2 * c]), lo_f(av[i][2 * c + 1]), hi_f(av[i][2 * c + 1]), sc);
                    store8(d, i & 1, i, k0, full_tag);
                    if (wc == 0) store_scale(sc, i, pcol0 / F8_BLOCK, full_tag);
                }
            } else {
                const int k0 = pcol0 + F8_BLOCK * wc, kb = k0 / F8_BLOCK;     // the wave's block of dA
                if (k0 < part_p) {
                    // the rows of h1, gate and up, of block (i, 64 columns jh)
                    uint4 hg[4], hu[4];
                    auto load_h1 = [&](int i, int jh) {
                        // rows that exist, from a uniform one on (32-bit offsets: 32 rows of 4 part bytes)
                        const int r0 = min(32 * BR * wr + 32 * i, prows - 1), last = prows - 1 - r0;
                        const int c = min(k0 + 64 * jh + chunk, p.n.part - 8);     // past the end: values that meet dA = 0
                        const uint16_t* gate = uni_ptr(p.h1 + static_cast<int64_t>(prow0 + r0) * 2 * p.n.part);
                        const uint16_t* up = uni_ptr(gate + p.n.part);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t at = static_cast<uint32_t>(min(8 * k + (ln >> 3), last)) * (2 * p.n.part) + c;
                            hg[k] = ld16_nt(gate + at);
                            hu[k] = ld16_nt(up + at);
                        }
                    };
                    auto put_rows = [&](const uint4 (&o)[4]) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(stg + (8 * k + (ln >> 3)) * 64 + (ln & 7) * 8) = o[k];
                    };
                    load_h1(0, 0);
                    static_for<BR>([&](auto i_tag) {
                        constexpr int i = decltype(i_tag)::value;
                        float v[2][2][16];      // [gate, up][64 columns]: pairs, kept where the block's sums were
                        uint32_t top[2] = {0, 0};
                        static_for<2>([&](auto jh_tag) {
                            constexpr int jh = decltype(jh_tag)::value;
                            uint2 d[8], g[8], u[8];
                            put_rows(hg);
                            take(g);
                            put_rows(hu);
                            take(u);
                            if constexpr (2 * i + jh + 1 < 2 * BR) load_h1((2 * i + jh + 1) / 2, (jh + 1) % 2);
                            sums(i_tag, jh_tag, d);
#pragma unroll
                            for (int c = 0; c < 8; ++c)
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const uint32_t dd = y ? d[c].y : d[c].x, gg = y ? g[c].y : g[c].x, uu = y ? u[c].y : u[c].x;
                                    float g0, u0, g1, u1;
                                    f8_act_grad(lo_f(gg), lo_f(uu), lo_f(dd), p.slope, e2, g0, u0);
                                    f8_act_grad(hi_f(gg), hi_f(uu), hi_f(dd), p.slope, e2, g1, u1);
                                    const uint32_t pg = pack2(g0, g1), pu = pack2(u0, u1);
                                    top[0] = f8_max2(top[0], pg);
                                    top[1] = f8_max2(top[1], pu);
                                    v[0][jh][2 * c + y] = acc_wr(pg);
                                    v[1][jh][2 * c + y] = acc_wr(pu);
                                }
                            fence();
                        });
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const F8Scale sc = f8_scale(max_other_half(f8_top(top[h])));
#pragma unroll
                            for (int jh = 0; jh < 2; ++jh) {
                                uint32_t d[8];
#pragma unroll
                                for (int c = 0; c < 8; ++c) {
                                    const uint32_t x = acc_rd_u(v[h][jh][2 * c]), y = acc_rd_u(v[h][jh][2 * c + 1]);
                                    d[c] = f8_four(lo_f(x), hi_f(x), lo_f(y), hi_f(y), sc);
                                }
                                store8(d, jh, i, h * part_p + k0 + 64 * jh, full_tag);
                            }
                            store_scale(sc, i, kb + h * (part_p / F8_BLOCK), full_tag);
                            fence();
                        }
                    });
                }
            }
        };
        if (full) epilogue(GrpTag<1>{});
        else epilogue(GrpTag<0>{});
        t += G;
        tile = next;
#pragma unroll
        for (int c = 0; c < WS; ++c) wd_next[c] = wd_first[c];
    }
    wait_vmcnt<0>();     // the last copies: none is under way to LDS that is another workgroup's
    if (p.group == 0) return;
    __syncthreads();
    f8_stream_list<EPI, FP32>(p, s_off, s_pre, s_ring, reinterpret_cast<uint32_t(*)[4][F8_GROUP]>(s_stg));
}

// ---------------------------------------------------------------- launchers
template <int MODE, int U>
static hipError_t launch_quant(const F8QuantParams& p, int num_cu, hipStream_t s) {
    const int width = MODE == F8_DGLU ? p.dim.part_p : p.dim.padded();
    const int64_t gy = (width + 512 * U - 1) / (512 * U);
    const int64_t want = (static_cast<int64_t>(p.M) / 2 + 1 + 3) / 4, most = (static_cast<int64_t>(num_cu) * 64 + gy - 1) / gy;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most), static_cast<unsigned>(gy));
    hipLaunchKernelGGL((f8_quant_kernel<MODE, U>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_f8_quant(F8Mode mode, const F8QuantParams& p, int num_cu, hipStream_t s) {
    // few rows: a group of columns a wave, for more waves
    const bool few = static_cast<int64_t>(p.M) < 16 * num_cu;
    switch (mode) {
        case F8_PLAIN: return few ? launch_quant<F8_PLAIN, 1>(p, num_cu, s) : launch_quant<F8_PLAIN, 4>(p, num_cu, s);
        case F8_GLU: return few ? launch_quant<F8_GLU, 1>(p, num_cu, s) : launch_quant<F8_GLU, 2>(p, num_cu, s);
        default: return launch_quant<F8_DGLU, 1>(p, num_cu, s);
    }
}

hipError_t launch_f8_quant_weights(const uint16_t* w, int E, const F8Dim& n, const F8Dim& k, uint8_t* q, uint8_t* s,
                                   hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(n.blocks() * k.blocks()), static_cast<unsigned>(E));    // at most 2^17, 2^10
    hipLaunchKernelGGL(f8_quant_weights_kernel, grid, dim3(256), 0, stream, w, n, k, q, s);
    return hipGetLastError();
}

hipError_t launch_f8_pack(const uint8_t* q, const uint8_t* s, int E, const F8Dim& n, const F8Dim& k, int transposed,
                          uint8_t* packed, hipStream_t stream) {
    const int64_t bytes = E * f8_matrix_bytes(n, k);
    int64_t blocks = (bytes / 16 + 255) / 256;
    if (blocks > 65536) blocks = 65536;
    hipLaunchKernelGGL(f8_pack_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, q, s, E, n, k, transposed,
                       packed, packed + bytes);
    return hipGetLastError();
}

template <int BR, int BC, int EPI, int FP32>
static hipError_t launch_tiles(const F8Params& p, int num_cu, hipStream_t s) {
    constexpr int TR = 64 * BR, OC = EPI == F8_STORE_GLU ? 32 * BC : 64 * BC;
    const int width = EPI == F8_STORE_GLU ? p.n.part_p : p.n.padded();
    const int64_t upper = (static_cast<int64_t>(p.M) / TR + (p.M < p.E ? p.M : p.E)) * ((width + OC - 1) / OC);
    const dim3 grid(static_cast<unsigned>(upper < num_cu && p.group == 0 ? upper : num_cu));
    hipLaunchKernelGGL((f8_tile_kernel<BR, BC, EPI, FP32>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <int EPI, int FP32>
static hipError_t launch_gemm(const F8Params& p, int num_cu, hipStream_t s) {
    F8Params g = p;
    const int blocks = EPI == F8_STORE_GLU ? p.n.part_p / F8_BLOCK : p.n.blocks();
    const F8Plan plan = f8_plan(p.M, p.E, EPI == F8_STORE_GLU ? blocks : (blocks + 1) / 2, EPI == F8_STORE ? blocks : 0,
                                p.kblocks, num_cu);
    g.tile = plan.rows != 0;
    g.group = plan.group;
    if (plan.rows == 256) return launch_tiles<4, 4, EPI, FP32>(g, num_cu, s);
    if (plan.rows && plan.columns == 256) return launch_tiles<2, 4, EPI, FP32>(g, num_cu, s);
    if (plan.rows) {
        if constexpr (EPI == F8_STORE) return launch_tiles<2, 2, EPI, FP32>(g, num_cu, s);
    }
    const int64_t groups = static_cast<int64_t>(p.M) / g.group + (p.M < p.E ? p.M : p.E);
    const int64_t upper = groups * blocks;
    hipLaunchKernelGGL((f8_stream_kernel<EPI, FP32>), dim3(static_cast<unsigned>(upper < num_cu ? upper : num_cu)), dim3(256), 0, s, g);
    return hipGetLastError();
}

hipError_t launch_f8_gemm(F8Epilogue epilogue, const F8Params& p, int num_cu, hipStream_t s) {
    switch (epilogue) {
        case F8_STORE: return p.fp32_sums ? launch_gemm<F8_STORE, 1>(p, num_cu, s) : launch_gemm<F8_STORE, 0>(p, num_cu, s);
        case F8_STORE_GLU: return p.fp32_sums ? launch_gemm<F8_STORE_GLU, 1>(p, num_cu, s) : launch_gemm<F8_STORE_GLU, 0>(p, num_cu, s);
        default: return p.fp32_sums ? launch_gemm<F8_STORE_DGLU, 1>(p, num_cu, s) : launch_gemm<F8_STORE_DGLU, 0>(p, num_cu, s);
    }
}

}  // namespace gg
