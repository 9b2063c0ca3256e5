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
// Non-temporal 16-byte accesses, for rows that a launch moves once: on MI355X
// a kernel that reads two and writes one 1 GiB array moves 5.1 TB/s with plain
// accesses, 5.5 with non-temporal stores and 5.9 with both.
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
__device__ __forceinline__ uint4 ld16_nt(const void* p) {
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load(static_cast<const u32x4*>(p)));
}
__device__ __forceinline__ void st16_nt(void* p, uint4 v) {
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), static_cast<u32x4*>(p));
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

// The same by a whole wave: every lane looks at every 64th expert.
__device__ __forceinline__ int find_expert_wave(const int* s_pre, int E, int t) {
    int below = 0;   // experts with s_pre <= t, which come first
    for (int e = threadIdx.x & 63; e - static_cast<int>(threadIdx.x & 63) < E; e += 64)
        below += __builtin_popcountll(__ballot(e < E && s_pre[min(e, E - 1)] <= t));
    return below - 1;
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

// Inclusive scan over the 64 lanes (v >= 0; op: sum or maximum) by the DPP
// row shifts and row broadcasts, without LDS.
template <typename Op>
__device__ __forceinline__ int wave_scan(int v, Op op) {
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));   // row_shr:1
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));   // row_shr:2
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));   // row_shr:4
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));   // row_shr:8
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));   // row_bcast:15 into rows 1 and 3
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));   // row_bcast:31 into rows 2 and 3
    return v;
}
// The value of the lane before (0 in lane 0), given an inclusive scan's values.
__device__ __forceinline__ int lane_before(int v) {
    return __builtin_amdgcn_update_dpp(0, v, 0x138, 0xf, 0xf, false);       // wave_shr:1
}

// Offsets of a chunk of 256 experts, four a lane (o[j]: first row of expert
// base + 4 lane + j, o[4]: its successor's), clamped into [0, M] and made
// non-decreasing by a running maximum (`top` carries it between chunks), so
// that bad offsets cannot count more rows than M.  Experts past E have no rows.
constexpr int EXPERT_CHUNK = 256;
__device__ __forceinline__ void load_offsets(const int64_t* __restrict__ offsets, int E, int M, int base, int& top,
                                             int (&o)[5]) {
    const int e0 = base + 4 * (threadIdx.x & 63);
#pragma unroll
    for (int j = 0; j < 5; ++j) {
        const int64_t v = offsets[min(e0 + j, E)];
        o[j] = static_cast<int>(v < 0 ? 0 : (v > M ? M : v));
    }
#pragma unroll
    for (int j = 1; j < 5; ++j) o[j] = max(o[j], o[j - 1]);
    const int incl = wave_scan(o[4], [](int a, int b) { return max(a, b); });
    const int before = max(lane_before(incl), top);
#pragma unroll
    for (int j = 0; j < 5; ++j) o[j] = max(o[j], before);
    top = max(top, __builtin_amdgcn_readlane(incl, 63));
}

// Exclusive prefix sums of count(rows of e) over the experts, and the offsets,
// into LDS (every thread of the workgroup calls it).
template <typename F>
__device__ __forceinline__ void prefix_experts(const int64_t* __restrict__ offsets, int E, int M, int* s_off,
                                               int* s_pre, F&& count) {
    if (threadIdx.x < 64) {
        int top = 0, sum = 0;
        for (int base = 0; base <= E; base += EXPERT_CHUNK) {
            int o[5], c[4];
            load_offsets(offsets, E, M, base, top, o);
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = count(o[j + 1] - o[j]);
            const int incl = wave_scan(c[0] + c[1] + c[2] + c[3], [](int a, int b) { return a + b; });
            int run = sum + lane_before(incl);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = base + 4 * threadIdx.x + j;
                if (e <= E) {
                    s_off[e] = o[j];
                    s_pre[e] = run;
                }
                run += c[j];
            }
            sum += __builtin_amdgcn_readlane(incl, 63);
        }
    }
    __syncthreads();
}

// The expert that owns item `target` of a list with count(rows)[0] items for
// each expert, its rows [lo, hi), and the sums of the NC counts over the
// experts before it; e = -1 past the end of the list.  Every wave finds it by
// itself, in registers, in the order of the offsets.
template <int NC>
struct ExpertItem {
    int e, lo, hi, before[NC];
};
template <int NC>
struct Counts {
    int c[NC];
};
template <int NC, typename F>
__device__ __forceinline__ ExpertItem<NC> find_item(const int64_t* __restrict__ offsets, int E, int M, int target,
                                                    F&& count) {
    ExpertItem<NC> item;
    item.e = -1;
    int top = 0, sum[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) sum[k] = 0;
    for (int base = 0; base < E; base += EXPERT_CHUNK) {
        int o[5], run[NC];
        Counts<NC> c[4];
        load_offsets(offsets, E, M, base, top, o);
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = count(o[j + 1] - o[j]);
        int total[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int incl = wave_scan(c[0].c[k] + c[1].c[k] + c[2].c[k] + c[3].c[k], [](int a, int b) { return a + b; });
            run[k] = sum[k] + lane_before(incl);
            total[k] = __builtin_amdgcn_readlane(incl, 63);
        }
        if (target < sum[0] + total[0]) {
            // the lane's expert that holds the target, if any (counts are zero or more, so it is unique)
            int at = -1;
            ExpertItem<NC> mine = {};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (run[0] <= target && target < run[0] + c[j].c[0]) {
                    at = j;
                    mine.lo = o[j];
                    mine.hi = o[j + 1];
#pragma unroll
                    for (int k = 0; k < NC; ++k) mine.before[k] = run[k];
                }
#pragma unroll
                for (int k = 0; k < NC; ++k) run[k] += c[j].c[k];
            }
            const int lane = __builtin_ctzll(__ballot(at >= 0));
            item.e = base + 4 * lane + __builtin_amdgcn_readlane(at, lane);
            item.lo = __builtin_amdgcn_readlane(mine.lo, lane);
            item.hi = __builtin_amdgcn_readlane(mine.hi, lane);
#pragma unroll
            for (int k = 0; k < NC; ++k) item.before[k] = __builtin_amdgcn_readlane(mine.before[k], lane);
            return item;
        }
#pragma unroll
        for (int k = 0; k < NC; ++k) sum[k] += total[k];
    }
    return item;
}

}  // namespace gg
