// Device helpers shared by the kernel files: bf16 conversion and packing,
// memory waits and barriers, LDS-DMA copies, and the prefix sums over experts
// that turn a work item's number into its expert.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gg {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) short i16x4;
typedef __attribute__((ext_vector_type(16))) float f32x16;

#define GG_AS3(p) ((__attribute__((address_space(3))) void*)(p))

__device__ __forceinline__ uint16_t f2bf(float f) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}
__device__ __forceinline__ float bf2f(uint32_t b16) {
    return __builtin_bit_cast(float, b16 << 16);
}
// Two floats rounded to bf16 (round to nearest even, as f2bf) and packed,
// lo in bits 0..15: one v_cvt_pk_bf16_f32 for the pair.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
// The same bits from two separate conversions.  Only one float is live at a
// time, which suits kernels short of registers (the eight-wave dgrad
// instances measured about 5% slower with the paired form).
__device__ __forceinline__ uint32_t pack2_sep(float lo, float hi) {
    return static_cast<uint32_t>(f2bf(lo)) | (static_cast<uint32_t>(f2bf(hi)) << 16);
}
// The two bf16 values of a packed pair as floats.
__device__ __forceinline__ float lo_f(uint32_t pr) { return __builtin_bit_cast(float, pr << 16); }
__device__ __forceinline__ float hi_f(uint32_t pr) { return __builtin_bit_cast(float, pr & 0xffff0000u); }

// Wait until at most N vector-memory operations of this wave are outstanding.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
    asm volatile("" ::: "memory");
}
// Workgroup barrier for the copy pipeline.  It first waits for this wave's
// outstanding LDS operations: a fragment read issued before the barrier must
// have completed before another wave refills that stage slot with LDS-DMA.
// (Outstanding HBM->LDS copies are waited for explicitly with wait_vmcnt.)
__device__ __forceinline__ void block_barrier() {
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0); the builtin keeps the compiler's count in step
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Wait states between the last MFMA and the first read of its accumulators.
// The compiler cannot count them where the read is inline assembly or where
// a branch skipped the last MFMA, so the epilogues issue them explicitly
// (24, more than a 16-pass MFMA needs).
__device__ __forceinline__ void mfma_drain() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
template <typename T>
__device__ __forceinline__ const T* uni_ptr(const T* ptr) {
    const uint64_t v = reinterpret_cast<uint64_t>(ptr);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return reinterpret_cast<const T*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// One wave-wide LDS-DMA load: every lane copies 16 bytes from base + voff
// (base wave-uniform, voff a per-lane 32-bit byte offset) to LDS byte address
// lds + 16 * lane (lds wave-uniform).  Issued from
// inline assembly so that the compiler does not add a conservative wait for
// all outstanding loads before every LDS read; the pipeline waits for the
// stage it needs explicitly (wait_vmcnt + barrier).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const void* base, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(voff), "s"(uni_ptr(base)), "s"(uni(lds)) : "memory", "m0");
}
// The same copy marked non-temporal (low retention in the caches), for data
// read once per pass: the streamed weights of the streaming items, which
// would otherwise push out of L2 the token panels that every item re-reads.
__device__ __forceinline__ void dma16_nt(const void* base, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1 nt"
                 :: "v"(voff), "s"(uni_ptr(base)), "s"(uni(lds)) : "memory", "m0");
}
#pragma clang diagnostic pop

// Read one accumulator register in the epilogue.  The accumulators live in
// AGPRs; reading them one at a time where they are consumed keeps the
// compiler from copying all of them to VGPRs at once at the end of the K loop.
__device__ __forceinline__ float acc_rd(float a) {
    float v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
    return v;
}
template <typename T>
__device__ __forceinline__ uint32_t lds_addr(const T* p) {
    return __builtin_amdgcn_readfirstlane(
        static_cast<uint32_t>(reinterpret_cast<uintptr_t>(GG_AS3(const_cast<T*>(p)))));
}

// Largest e in [0, E-1] with s_pre[e] <= t (t < s_pre[E]); skips empty experts.
__device__ __forceinline__ int find_expert(const int* s_pre, int E, int t) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_pre[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <int V> struct GrpTag { static constexpr int value = V; };
// f(GrpTag<0>{}), ..., f(GrpTag<N - 1>{}): a loop over compile-time indices.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    if constexpr (I < N) {
        f(GrpTag<I>{});
        static_for<N, I + 1>(f);
    }
}

// Exclusive prefix sums of count(rows of e) over the experts, and the offsets
// (every thread of the workgroup calls it).  The offsets are clamped into
// [0, M] and made non-decreasing by a running maximum, so bad offsets cannot
// count more rows than M.
template <typename F>
__device__ __forceinline__ void prefix_experts(const int64_t* __restrict__ offsets, int E, int M, int* s_off,
                                               int* s_pre, F&& count) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) {
        int64_t o = offsets[e];
        o = o < 0 ? 0 : (o > M ? M : o);
        s_off[e] = static_cast<int>(o);
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x, per = E / 64 + 1;
        const int e0 = min(E + 1, lane * per), e2 = min(E + 1, e0 + per), e1 = min(E, e2);
        int top = 0;
        for (int e = e0; e < e2; ++e) {
            top = max(top, s_off[e]);
            s_off[e] = top;
        }
        int before = __shfl_up(top, 1, 64);
        if (lane == 0) before = 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(before, d, 64);
            if (lane >= d) before = max(before, v);
        }
        for (int e = e0; e < e2; ++e) s_off[e] = max(s_off[e], before);
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the next lane's first offset
        int sum = 0;
        for (int e = e0; e < e1; ++e) sum += count(s_off[e + 1] - s_off[e]);
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(incl, d, 64);
            if (lane >= d) incl += v;
        }
        int run = incl - sum;
        for (int e = e0; e < e1; ++e) {
            s_pre[e] = run;
            run += count(s_off[e + 1] - s_off[e]);
        }
        if (lane == 63) s_pre[E] = incl;
    }
    __syncthreads();
}

}  // namespace gg
