// Entry points of the products with 4-bit weights: checks, and the choice of
// the kernel.
#include "qlin_w4.h"

namespace qlin {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 24;
constexpr int64_t kMaxW4K = (int64_t)1 << 20;
constexpr int64_t kMaxStride = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxRowBytes = (int64_t)1 << 25;        // of X and B: a workgroup's 64 rows lie within 2^31

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Checks shared by the two entry points; M is rows (a bound for experts).
qlin_status check(int64_t M, int64_t N, int64_t K, int64_t group, const void *X, int64_t ldx,
                  const void *B, int64_t ldb, qlin_scale_type st, const void *scale, const void *Y,
                  int64_t ldy)
{
    if (M < 0 || M > kMaxRows || N < 0 || N > kMaxRows || K <= 0 || K > kMaxW4K)
        return QLIN_ERR_BAD_SHAPE;
    if ((group != 32 && group != 64 && group != 128) ||
        (st != QLIN_SCALE_F32 && st != QLIN_SCALE_BF16 && st != QLIN_SCALE_F16))
        return QLIN_ERR_BAD_ARGUMENT;
    if (K % group != 0)
        return QLIN_ERR_BAD_SHAPE;
    if (M == 0 || N == 0)
        return QLIN_OK;
    if (!X || !B || !scale || !Y)
        return QLIN_ERR_NULL_POINTER;
    if (ldx < K || ldx % 8 != 0 || 2 * ldx > kMaxRowBytes || ldb < K / 2 || ldb % 16 != 0 ||
        ldb > kMaxRowBytes ||
        ldy < N || ldy > kMaxStride)
        return QLIN_ERR_BAD_STRIDE;
    if (!aligned(X, 16) || !aligned(B, 16) || !aligned(Y, 16) || !aligned(scale, 4))
        return QLIN_ERR_MISALIGNED;
    return QLIN_OK;
}

w4::Args make_args(int64_t M, int64_t N, int64_t K, int64_t group, const uint16_t *X, int64_t ldx,
                 const uint8_t *B, int64_t ldb, qlin_scale_type st, const void *scale,
                 const uint8_t *zero, uint16_t *Y, int64_t ldy)
{
    w4::Args a{};
    a.x = X;
    a.b = B;
    a.scale = static_cast<const uint8_t *>(scale);
    a.zero = zero;
    a.y = Y;
    a.ldx = ldx;
    a.ldb = ldb;
    a.ldy = ldy;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.G = (int)(K / group);
    a.st = (int)st;
    return a;
}

// Sum of the parts of K, in order; four outputs a thread where N allows, four
// parts on their way at a time (a launch and the latencies bound it: twelve parts of
// 32 x 5120 5 us under the profiler; ten were 4.3 us, one part after another 5.4).
template <int V>
__global__ void __launch_bounds__(256) k_reduce(w4::Args a)
{
    const int64_t all = (int64_t)a.M * a.N;
    const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
    const bool there = e < all;                     // (V divides N: all of the V, or none)
    constexpr int kAtOnce = 4;
    float v[V] = {};
    for (int s = 0; s < a.splits; s += kAtOnce) {
        float p[kAtOnce][V];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (there && s + j < a.splits)
                __builtin_memcpy(p[j], a.part + (s + j) * all + e, 4 * V);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (there && s + j < a.splits)
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] += p[j][i];
    }
    const int m = (int)(e / a.N), n = (int)(e % a.N);
#pragma unroll
    for (int i = 0; i < V; ++i) w4::store_value(a, there, m, n + i, v[i]);
}

size_t part_bytes(int64_t M, int64_t N, int splits) { return splits > 1 ? (size_t)splits * M * N * sizeof(float) : 0; }

qlin_status status_of(hipError_t e)
{
    return e == hipSuccess ? QLIN_OK : e == hipErrorInvalidConfiguration ? QLIN_ERR_BAD_SHAPE : QLIN_ERR_HIP;
}

qlin_status launch(w4::Args &a, void *ws, size_t ws_bytes, void *stream)
{
    static const w4::Launch kStream[3] = {w4::launch_stream_32, w4::launch_stream_64, w4::launch_stream_128};
    static const w4::Launch kTile[3] = {w4::launch_tile_32, w4::launch_tile_64, w4::launch_tile_128};
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int group = a.K / a.G, which = group == 128 ? 2 : group == 64 ? 1 : 0;
    a.splits = 1;
    a.split_k = a.K;
    if (w4::streams(a.M, a.N, a.experts, a.rows))
        return status_of(kStream[which](a, s));
    const w4::TilePick p = w4::pick_tile(a.M, a.N, a.K, a.experts, a.rows);
    const size_t need = part_bytes(a.M, a.N, p.splits);
    if (need && (!ws || ws_bytes < need))
        return QLIN_ERR_WORKSPACE;
    if (need && !aligned(ws, 16))
        return QLIN_ERR_MISALIGNED;
    const int stages = (a.K + p.ks - 1) / p.ks;
    a.tb = p.tb;
    a.rb = p.rb;
    a.splits = p.splits;
    a.split_k = (stages + p.splits - 1) / p.splits * p.ks;
    a.part = static_cast<float *>(ws);
    const qlin_status st = status_of(kTile[which](a, s));
    if (st != QLIN_OK)
        return st;
    if (a.splits > 1) {
        const int v = a.N % 4 == 0 ? 4 : 1;
        const dim3 grid((unsigned)(((int64_t)a.M * a.N / v + 255) / 256));
        if (v == 4)
            hipLaunchKernelGGL(k_reduce<4>, grid, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL(k_reduce<1>, grid, dim3(256), 0, s, a);
        if (hipGetLastError() != hipSuccess)
            return QLIN_ERR_HIP;
    }
    return QLIN_OK;
}

}  // namespace

}  // namespace qlin

using namespace qlin;

extern "C" {

qlin_status qlin_w4_mm(int64_t M, int64_t N, int64_t K, int64_t group, const uint16_t *X,
                       int64_t ldx, const uint8_t *B, int64_t ldb, qlin_scale_type st,
                       const void *b_scale, const uint8_t *b_zero, uint16_t *Y, int64_t ldy,
                       void *workspace, size_t workspace_bytes, void *stream)
{
    const qlin_status r = check(M, N, K, group, X, ldx, B, ldb, st, b_scale, Y, ldy);
    if (r != QLIN_OK || M == 0 || N == 0)
        return r;
    w4::Args a = make_args(M, N, K, group, X, ldx, B, ldb, st, b_scale, b_zero, Y, ldy);
    return launch(a, workspace, workspace_bytes, stream);
}

size_t qlin_w4_workspace_size(int64_t M, int64_t N, int64_t K)
{
    if (M <= 0 || M > kMaxRows || N <= 0 || N > kMaxRows || K <= 0 || K > kMaxW4K)
        return 0;
    return M <= w4::kStreamTokens ? 0 : part_bytes(M, N, w4::pick_tile(M, N, K, 0, 0).splits);
}

qlin_status qlin_grouped_w4_mm(int64_t groups, const int32_t *group_offsets, int64_t max_rows,
                               int64_t rows, int64_t N, int64_t K, int64_t group,
                               const uint16_t *X, int64_t ldx, const uint8_t *B, int64_t ldb,
                               int64_t b_group_stride, qlin_scale_type st, const void *b_scale,
                               const uint8_t *b_zero, uint16_t *Y, int64_t ldy, void *stream)
{
    if (groups < 0 || groups > 65535 || rows < 0 || rows > kMaxRows || max_rows < 0)
        return QLIN_ERR_BAD_SHAPE;
    const int64_t M = max_rows < rows ? max_rows : rows;
    const qlin_status r = check(groups ? M : 0, N, K, group, X, ldx, B, ldb, st, b_scale, Y, ldy);
    if (r != QLIN_OK || groups == 0 || M == 0 || N == 0)
        return r;
    if (!group_offsets)
        return QLIN_ERR_NULL_POINTER;
    if (b_group_stride < 0 || b_group_stride % 16 != 0)
        return QLIN_ERR_BAD_STRIDE;
    if (!aligned(group_offsets, 4))
        return QLIN_ERR_MISALIGNED;
    w4::Args a = make_args(M, N, K, group, X, ldx, B, ldb, st, b_scale, b_zero, Y, ldy);
    a.group_off = group_offsets;
    a.b_gstride = b_group_stride;
    a.rows = (int)rows;
    a.experts = (int)groups;
    return launch(a, nullptr, 0, stream);
}

}  // extern "C"
