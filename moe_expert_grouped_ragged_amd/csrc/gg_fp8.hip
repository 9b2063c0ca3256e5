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
// The largest |v| of a packed pair of bf16 values, as fp32 bits.
__device__ __forceinline__ uint32_t f8_top2(uint32_t pair) {
    return max((pair & 0x7fffu) << 16, pair & 0x7fff0000u);
}

// The activation and its derivative on bf16 values, with the arithmetic of the
// bf16 path's epilogues: A = bf16(act(gate) * up), dH1 = bf16 of dg and du.
__device__ __forceinline__ float f8_act(float g, float u, float slope) {
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-(slope * g))) * u;
}
__device__ __forceinline__ void f8_act_grad(float g, float u, float da, float slope, float& dg, float& du) {
    const float sg = __builtin_amdgcn_rcpf(1.0f + __expf(-(slope * g)));
    dg = da * u * sg * (1.0f + slope * g * (1.0f - sg));
    du = da * g * sg;
}

// Half a wave takes 512 columns of a row, 16 a lane, so eight lanes are a block
// and its maximum stays in registers; the two halves take neighbouring rows
// from an even one on, so that a store covers whole 128-byte lines of the two
// rows in the product's layout.  U such groups of columns are in flight at a
// time.  Bound by the bytes.
template <int MODE, int U>
__global__ __launch_bounds__(256) void f8_quant_kernel(const F8QuantParams p) {
    constexpr int PARTS = MODE == F8_DGLU ? 2 : 1;    // blocks that a lane makes at a time
    constexpr int IN = MODE == F8_PLAIN ? 1 : (MODE == F8_GLU ? 2 : 3);
    const int lane = threadIdx.x & 63, sub = lane & 31;
    const auto clamp = [&](int64_t o) { return static_cast<int>(o < 0 ? 0 : (o > p.M ? p.M : o)); };
    const int lo = clamp(p.offsets[0]), hi = clamp(p.offsets[p.E]);
    const int part = p.dim.part, part_p = p.dim.part_p;
    const int width = MODE == F8_DGLU ? part_p : p.dim.padded();
    const int64_t qblock = static_cast<int64_t>(p.M) * 64;
    for (int64_t r0 = (lo & ~1) + 2 * (static_cast<int64_t>(blockIdx.x) * 4 + uni(threadIdx.x >> 6)); r0 < hi;
         r0 += static_cast<int64_t>(gridDim.x) * 8) {
        const int64_t r = r0 + (lane >> 5);
        const bool live = r >= lo && r < hi;
        const int64_t rr = live ? r : (r < lo ? r + 1 : r - 1);    // a row that exists, where this half has none
        uint4 in[U][IN][2];
        const int c0 = (static_cast<int>(blockIdx.y) * U) * 512 + sub * 16;
        // the real column of a padded one's 16, and whether its two eights exist
        auto at = [&](int u, bool (&ok)[2]) {
            const int c = c0 + u * 512;
            const int h = MODE != F8_DGLU && c >= part_p, k = c - h * part_p;
            ok[0] = c < width && k < part;
            ok[1] = c < width && k + 8 < part;
            return h * part + k;
        };
#pragma unroll
        for (int u = 0; u < U; ++u) {
            bool ok[2];
            const int col = at(u, ok);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < IN; ++i) in[u][i][e] = zero;
                if (!ok[e]) continue;
                if constexpr (MODE == F8_PLAIN) {
                    in[u][0][e] = ld16_nt(p.x + rr * p.dim.real() + col + 8 * e);
                } else {
                    const uint16_t* h = (MODE == F8_GLU ? p.x : p.h1) + rr * 2 * part + col + 8 * e;
                    in[u][0][e] = ld16_nt(h);
                    in[u][1][e] = ld16_nt(h + part);
                    if constexpr (MODE == F8_DGLU) in[u][IN - 1][e] = ld16_nt(p.x + rr * part + col + 8 * e);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            bool ok[2];
            const int col = at(u, ok);
            const int c = c0 + u * 512;
            if (c >= width) continue;     // whole blocks of lanes
            uint32_t v[PARTS][8];         // 16 bf16 values
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint4(&x)[IN][2] = in[u];
                const uint32_t a[4] = {x[0][e].x, x[0][e].y, x[0][e].z, x[0][e].w};
                const uint32_t b[4] = {x[IN > 1][e].x, x[IN > 1][e].y, x[IN > 1][e].z, x[IN > 1][e].w};
                const uint32_t d[4] = {x[IN - 1][e].x, x[IN - 1][e].y, x[IN - 1][e].z, x[IN - 1][e].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (MODE == F8_PLAIN) {
                        v[0][4 * e + i] = a[i];
                    } else if constexpr (MODE == F8_GLU) {
                        v[0][4 * e + i] = pack2(f8_act(lo_f(a[i]), lo_f(b[i]), p.slope), f8_act(hi_f(a[i]), hi_f(b[i]), p.slope));
                    } else {
                        float g0, u0, g1, u1;
                        f8_act_grad(lo_f(a[i]), lo_f(b[i]), lo_f(d[i]), p.slope, g0, u0);
                        f8_act_grad(hi_f(a[i]), hi_f(b[i]), hi_f(d[i]), p.slope, g1, u1);
                        v[0][4 * e + i] = pack2(g0, g1);
                        v[PARTS - 1][4 * e + i] = pack2(u0, u1);
                    }
                }
                if constexpr (MODE != F8_PLAIN) {
                    if (p.v_out && live && ok[e]) {
                        uint16_t* o = p.v_out + r * p.dim.real() + col + 8 * e;
#pragma unroll
                        for (int h = 0; h < PARTS; ++h)
                            st16_nt(o + h * part, make_uint4(v[h][4 * e], v[h][4 * e + 1], v[h][4 * e + 2], v[h][4 * e + 3]));
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < PARTS; ++h) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, f8_top2(v[h][i]));
                m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0xb1, 0xf, 0xf, true)));    // lane ^ 1
                m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x4e, 0xf, 0xf, true)));    // lane ^ 2
                m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x141, 0xf, 0xf, true)));   // the other four
                const F8Scale s = f8_scale(m);
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = f8_four(lo_f(v[h][2 * i]), hi_f(v[h][2 * i]), lo_f(v[h][2 * i + 1]), hi_f(v[h][2 * i + 1]), s);
                if (!live) continue;
                const int cp = c + h * part_p, kb = cp / F8_BLOCK;
                *reinterpret_cast<uint4*>(p.q + (cp >> 6) * qblock + r * 64 + (cp & 63)) = make_uint4(o[0], o[1], o[2], o[3]);
                if ((lane & 7) == 0) p.s[4 * (static_cast<int64_t>(kb >> 2) * p.M + r) + (kb & 3)] = static_cast<uint8_t>(s.byte);
            }
        }
    }
}

// A workgroup a 128 x 128 block: 16 rows of 16 lanes of eight columns at a time, held in registers.
__global__ __launch_bounds__(256) void f8_quant_weights_kernel(const uint16_t* __restrict__ w, F8Dim n, F8Dim k,
                                                               uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
    __shared__ uint32_t s_top[4];
    const int64_t b = blockIdx.x;
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
        m = max(max(max(m, f8_top2(v[i].x)), max(f8_top2(v[i].y), f8_top2(v[i].z))), f8_top2(v[i].w));
    }
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
            for (int j = 0; j < 16; ++j) {
                const int c = f8_real(cont, st * 64 + 32 * (l >> 5) + 16 * h + j);
                if (c < 0) continue;
                const uint8_t x = transposed ? m[static_cast<int64_t>(c) * K + row] : m[static_cast<int64_t>(row) * K + c];
                w[j >> 2] |= static_cast<uint32_t>(x) << (8 * (j & 3));
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
// out[r][n] = sum over blocks of 128 of 2^(s_r + s_w) sum q w: the matrix
// instruction multiplies by both scales, so the fp32 sums run over all blocks
// without a step between them.  The instruction adds eight neighbouring
// products at a time, each cut towards zero below 2^-13 of the power of two of
// the largest's factors, and joins these sums in fp32 (measured by planted
// values).  On normal data that is about 2^-13 of the result, where its
// rounding to bf16 is up to 2^-9 and the operands' to e4m3 2^-4; the
// instructions that keep all bits run at half the rate.  Every kernel adds a row's products in the same
// order (steps of 64 columns, one 32x32x64 instruction each), so a row's bits
// do not depend on the batch.
__device__ __forceinline__ f32x16 f8_mma(i32x8 w, i32x8 t, f32x16 acc, int ws, int ts) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, t, acc, 0, 0, 0, ws, 0, ts);
}
__device__ __forceinline__ i32x8 f8_join(i32x4 a, i32x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// One wave's 32 output columns (padded block nb) for up to 32 TB rows over the whole summed dimension, one block of
// 128 loaded while another is multiplied.
template <int TB>
__device__ __forceinline__ void f8_stream_block(const F8Params& p, const uint8_t* w, const uint8_t* ws, int row0, int rows,
                                                int nb) {
    const int lane = threadIdx.x & 63;
    const uint8_t* wp = w + static_cast<int64_t>(nb) * p.kblocks * 4096 + lane * 16;
    const uint8_t* sp = ws + static_cast<int64_t>(nb >> 2) * p.ws_ld;
    const uint8_t *tp[TB], *ts[TB];
#pragma unroll
    for (int i = 0; i < TB; ++i) {
        const int64_t r = row0 + min(i * 32 + (lane & 31), rows - 1);
        tp[i] = p.q + r * 64 + 32 * (lane >> 5);
        ts[i] = p.s + r * 4;
    }
    const int64_t block = static_cast<int64_t>(p.M) * 64, sgroup = static_cast<int64_t>(p.M) * 4;
    f32x16 acc[TB];
#pragma unroll
    for (int i = 0; i < TB; ++i) acc[i] = f32x16{};
    i32x4 wv[2][4], tv[2][TB][4];
    int wsv[2], tsv[2][TB];
    auto load = [&](auto buf_tag, int k) {
        constexpr int buf = decltype(buf_tag)::value;
        k = min(k, p.kblocks - 1);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            wv[buf][u] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(wp + static_cast<int64_t>(k) * 4096 + u * 1024));
        wsv[buf] = sp[k];
#pragma unroll
        for (int i = 0; i < TB; ++i) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                tv[buf][i][u] = *reinterpret_cast<const i32x4*>(tp[i] + (2 * k + (u >> 1)) * block + 16 * (u & 1));
            tsv[buf][i] = ts[i][(k >> 2) * sgroup + (k & 3)];
        }
    };
    auto mma = [&](auto buf_tag) {
        constexpr int buf = decltype(buf_tag)::value;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < TB; ++i)
                acc[i] = f8_mma(f8_join(wv[buf][2 * u], wv[buf][2 * u + 1]), f8_join(tv[buf][i][2 * u], tv[buf][i][2 * u + 1]),
                                acc[i], wsv[buf], tsv[buf][i]);
    };
    load(GrpTag<0>{}, 0);
    for (int k = 0; k < p.kblocks; k += 2) {
        load(GrpTag<1>{}, k + 1);
        mma(GrpTag<0>{});
        load(GrpTag<0>{}, k + 2);
        if (k + 1 < p.kblocks) mma(GrpTag<1>{});
    }
    // lane holds row lane & 31 of each 32-row block and, in register 4q + x, column 32 nb + 8q + 4(lane >> 5) + x
    const int h = nb * 32 >= p.n.part_p;
#pragma unroll
    for (int i = 0; i < TB; ++i) {
        const int r = i * 32 + (lane & 31);
        if (r >= rows) continue;
        uint16_t* orow = p.out + static_cast<int64_t>(row0 + r) * p.n.real() + h * p.n.part;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int n = nb * 32 - h * p.n.part_p + 8 * q + 4 * (lane >> 5);
            if (n < p.n.part)
                *reinterpret_cast<uint2*>(orow + n) = make_uint2(pack2(acc[i][4 * q], acc[i][4 * q + 1]),
                                                                 pack2(acc[i][4 * q + 2], acc[i][4 * q + 3]));
        }
    }
}

// The list of all (row group, 128-column block) pairs, groups of up to 96 rows, a workgroup an item and a wave 32
// of its columns.
constexpr int F8_GROUP = 96;

__global__ __launch_bounds__(256) void f8_stream_kernel(const F8Params p) {
    __shared__ int s_off[GG_KMAX_EXPERTS + 1];
    __shared__ int s_pre[GG_KMAX_EXPERTS + 1];
    const int nblocks = p.n.blocks();
    prefix_experts(p.offsets, p.E, p.M, s_off, s_pre, [&](int m) { return (m + F8_GROUP - 1) / F8_GROUP * nblocks; });
    const int total = uni(s_pre[p.E]);
    const int wave = uni(threadIdx.x >> 6);
    for (int it = blockIdx.x; it < total; it += gridDim.x) {
        const int e = uni(find_expert_wave(s_pre, p.E, it));
        const int local = it - uni(s_pre[e]), grp = local / nblocks, nb = (local - grp * nblocks) * 4 + wave;
        const int row0 = uni(s_off[e]) + grp * F8_GROUP, rows = min(F8_GROUP, uni(s_off[e + 1]) - row0);
        const uint8_t* w = p.w + static_cast<int64_t>(e) * p.w_stride;
        const uint8_t* ws = p.ws + static_cast<int64_t>(e) * p.ws_stride;
        const int tb = (rows + 31) / 32;
        if (tb == 1) f8_stream_block<1>(p, w, ws, row0, rows, nb);
        else if (tb == 2) f8_stream_block<2>(p, w, ws, row0, rows, nb);
        else f8_stream_block<3>(p, w, ws, row0, rows, nb);
    }
}

// ---------------------------------------------------------------- launchers
template <int MODE, int U>
static hipError_t launch_quant(const F8QuantParams& p, int num_cu, hipStream_t s) {
    const int width = MODE == F8_DGLU ? p.dim.part_p : p.dim.padded();
    const int64_t gy = (width + 512 * U - 1) / (512 * U);
    const int64_t want = (static_cast<int64_t>(p.M) / 2 + 1 + 3) / 4, most = (static_cast<int64_t>(num_cu) * 16 + gy - 1) / gy;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most), static_cast<unsigned>(gy));
    hipLaunchKernelGGL((f8_quant_kernel<MODE, U>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_f8_quant(F8Mode mode, const F8QuantParams& p, int num_cu, hipStream_t s) {
    switch (mode) {
        case F8_PLAIN: return launch_quant<F8_PLAIN, 2>(p, num_cu, s);
        case F8_GLU: return launch_quant<F8_GLU, 1>(p, num_cu, s);
        default: return launch_quant<F8_DGLU, 1>(p, num_cu, s);
    }
}

hipError_t launch_f8_quant_weights(const uint16_t* w, int E, const F8Dim& n, const F8Dim& k, uint8_t* q, uint8_t* s,
                                   hipStream_t stream) {
    const int64_t blocks = static_cast<int64_t>(E) * n.blocks() * k.blocks();
    hipLaunchKernelGGL(f8_quant_weights_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, w, n, k, q, s);
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

hipError_t launch_f8_gemm(const F8Params& p, int num_cu, hipStream_t s) {
    const int64_t groups = static_cast<int64_t>(p.M) / F8_GROUP + (p.M < p.E ? p.M : p.E);
    const int64_t upper = groups * p.n.blocks(), most = static_cast<int64_t>(num_cu) * 3;
    hipLaunchKernelGGL(f8_stream_kernel, dim3(static_cast<unsigned>(upper < most ? upper : most)), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace gg
