// C-ABI entry points of the expert adapters: argument validation, workspace
// layout and launches.  Declarations and the contract are in include/gg.h.
//
// Every argument check runs before the first HIP call.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gg.h"
#include "gg_adapter.h"
#include "gg_host.h"

namespace {

using namespace gg;

int check_adapter_shape(int64_t M, int64_t E, int64_t N, int64_t K, int64_t r) {
    if (E < 1 || E > GG_MAX_EXPERTS) return GG_ERR_INVALID_ARGUMENT;
    if (N <= 0 || K <= 0 || N % 8 != 0 || K % 8 != 0 || N >= (int64_t(1) << 22) || K >= (int64_t(1) << 22))
        return GG_ERR_INVALID_ARGUMENT;
    if (r < 1 || r > GG_ADAPTER_MAX_RANK || M < 0 || M >= (int64_t(1) << 31)) return GG_ERR_INVALID_ARGUMENT;
    return GG_OK;
}

// Rows of a unit of a backward kernel whose workgroups each own one of
// `chunks` column chunks (about: an expert's rows are divided evenly): about
// `units` units when the rows are spread evenly,
// and at least 256 rows, so that the fp32 part a unit leaves behind stays
// small next to the rows it reads; at most 2^30, which the kernels count in 32 bits.
int64_t unit_rows(int64_t M, int64_t chunks, int64_t units) {
    const int64_t rows = (M * chunks / units + AD_BLK - 1) / AD_BLK * AD_BLK;
    return rows < 256 ? 256 : (rows < (int64_t(1) << 30) ? rows : int64_t(1) << 30);
}

// Workspace of the backward pass: byte offsets of its arrays.
struct Workspace {
    int64_t rows1, rows2, blocks;
    size_t du_part, du, du_t, db_part, da_part, total;
};

Workspace workspace_of(int64_t M, int64_t E, int64_t N, int64_t K, int64_t r) {
    Workspace w{};
    const int64_t rp = ad_rank_p(static_cast<int>(r));
    const int64_t chunks = ad_chunks(static_cast<int>(N), static_cast<int>(rp));
    // two workgroups of the smallest rank share a CU, and its parts are small (131072 rows, Zipf, N 2048:
    // rank 16 341 us, 360 us with half the units; rank 32 385 us, 437 us with twice as many)
    w.rows1 = unit_rows(M, chunks, rp == 16 ? 1024 : 512);
    w.rows2 = unit_rows(M, (K + 4 * AD_WCOLS - 1) / (4 * AD_WCOLS), 1024);
    w.blocks = M / AD_BLK + (M < E ? M : E);
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += (static_cast<size_t>(bytes) + 255) / 256 * 256;
        return here;
    };
    w.du_part = take(chunks * w.blocks * AD_BLK * rp * 4);
    w.du = take(w.blocks * AD_BLK * (rp < 32 ? 32 : rp) * 2);
    w.du_t = take(w.blocks * AD_BLK * rp * 6);
    // an expert of several units has at most m / rows + 1/2 of them, and at least 3/2 rows
    w.db_part = take(M > w.rows1 ? 2 * M / w.rows1 * N * r * 4 : 0);
    w.da_part = take(M > w.rows2 ? 2 * M / w.rows2 * K * r * 4 : 0);
    w.total = at;
    return w;
}

}  // namespace

extern "C" {

int gg_adapter_forward(const void* x, const int64_t* offsets, int64_t M, const void* a, const void* b, int64_t E,
                       int64_t N, int64_t K, int64_t r, float scale, const void* base, void* u, void* y,
                       hipStream_t stream) {
    int st = check_adapter_shape(M, E, N, K, r);
    if (st != GG_OK) return st;
    if (M == 0) return GG_OK;
    if (!x || !offsets || !a || !b || !u || !y) return GG_ERR_INVALID_ARGUMENT;
    if (!aligned16(x) || !aligned16(a) || !aligned16(b) || !aligned16(u) || !aligned16(y) || (base && !aligned16(base)) ||
        (reinterpret_cast<uintptr_t>(offsets) & 7u))
        return GG_ERR_MISALIGNED;
    const Range rbase = range_of(base, base && base != y ? M * N * 2 : 0);
    st = check_aliasing({range_of(x, M * K * 2), range_of(offsets, (E + 1) * 8), range_of(a, E * r * K * 2),
                         range_of(b, E * N * r * 2), rbase},
                        {range_of(y, M * N * 2), range_of(u, M * r * 2)});
    if (st != GG_OK) return st;
    DeviceInfo info;
    if ((st = device_info(stream, &info)) != GG_OK) return st;
    if ((st = debug_validate_offsets(offsets, E, M, stream)) != GG_OK) return st;
    AdapterParams p{};
    p.x = static_cast<const uint16_t*>(x);
    p.offsets = offsets;
    p.a = static_cast<const uint16_t*>(a);
    p.b = static_cast<const uint16_t*>(b);
    p.base = static_cast<const uint16_t*>(base);
    p.M = static_cast<int>(M);
    p.E = static_cast<int>(E);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.r = static_cast<int>(r);
    p.scale = scale;
    p.u = static_cast<uint16_t*>(u);
    p.out = static_cast<uint16_t*>(y);
    return launch_adapter_forward(p, info.num_cu, stream) == hipSuccess ? GG_OK : GG_ERR_HIP;
}

size_t gg_adapter_workspace_bytes(int64_t M, int64_t E, int64_t N, int64_t K, int64_t r) {
    if (M == 0 || check_adapter_shape(M, E, N, K, r) != GG_OK) return 0;
    return workspace_of(M, E, N, K, r).total;
}

int gg_adapter_backward(const void* dy, const void* x, const void* u, const int64_t* offsets, int64_t M, const void* a,
                        const void* b, int64_t E, int64_t N, int64_t K, int64_t r, float scale, const void* base,
                        void* workspace, size_t workspace_bytes, void* dx, float* da, float* db, int accumulate,
                        hipStream_t stream) {
    int st = check_adapter_shape(M, E, N, K, r);
    if (st != GG_OK) return st;
    if (!da || !db || !offsets) return GG_ERR_INVALID_ARGUMENT;
    if (M > 0 && (!dy || !x || !u || !a || !b || !workspace || !dx)) return GG_ERR_INVALID_ARGUMENT;
    if (!aligned16(da) || !aligned16(db) || (reinterpret_cast<uintptr_t>(offsets) & 7u)) return GG_ERR_MISALIGNED;
    if (M > 0 && (!aligned16(dy) || !aligned16(x) || !aligned16(u) || !aligned16(a) || !aligned16(b) ||
                  !aligned16(workspace) || !aligned16(dx) || (base && !aligned16(base))))
        return GG_ERR_MISALIGNED;
    const Workspace w = workspace_of(M, E, N, K, r);
    if (M > 0 && workspace_bytes < w.total) return GG_ERR_WORKSPACE_TOO_SMALL;
    const Range rbase = range_of(base, base && base != dx ? M * K * 2 : 0);
    st = check_aliasing({range_of(dy, M * N * 2), range_of(x, M * K * 2), range_of(u, M * r * 2),
                         range_of(offsets, (E + 1) * 8), range_of(a, M ? E * r * K * 2 : 0),
                         range_of(b, M ? E * N * r * 2 : 0), rbase},
                        {range_of(dx, M * K * 2), range_of(workspace, M ? w.total : 0), range_of(da, E * r * K * 4),
                         range_of(db, E * N * r * 4)});
    if (st != GG_OK) return st;
    DeviceInfo info;
    if ((st = device_info(stream, &info)) != GG_OK) return st;
    if ((st = debug_validate_offsets(offsets, E, M, stream)) != GG_OK) return st;
    char* ws = static_cast<char*>(workspace);
    AdapterParams p{};
    p.x = static_cast<const uint16_t*>(x);
    p.offsets = offsets;
    p.a = static_cast<const uint16_t*>(a);
    p.b = static_cast<const uint16_t*>(b);
    p.base = static_cast<const uint16_t*>(base);
    p.M = static_cast<int>(M);
    p.E = static_cast<int>(E);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.r = static_cast<int>(r);
    p.scale = scale;
    p.u = const_cast<uint16_t*>(static_cast<const uint16_t*>(u));   // only read by the backward kernels
    p.out = static_cast<uint16_t*>(dx);
    p.dy = static_cast<const uint16_t*>(dy);
    p.da = da;
    p.db = db;
    p.accumulate = accumulate != 0;
    p.rows1 = static_cast<int>(w.rows1);
    p.rows2 = static_cast<int>(w.rows2);
    p.blocks = w.blocks;
    if (M > 0) {
        p.du_part = reinterpret_cast<float*>(ws + w.du_part);
        p.du = reinterpret_cast<uint16_t*>(ws + w.du);
        p.du_t = reinterpret_cast<uint16_t*>(ws + w.du_t);
        p.db_part = reinterpret_cast<float*>(ws + w.db_part);
        p.da_part = reinterpret_cast<float*>(ws + w.da_part);
    }
    return launch_adapter_backward(p, info.num_cu, stream) == hipSuccess ? GG_OK : GG_ERR_HIP;
}

}  // extern "C"
