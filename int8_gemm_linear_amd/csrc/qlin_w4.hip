// Entry points of the products with 4-bit weights: checks, and the choice of
// the kernel.
#include "qlin_w4.h"

namespace qlin {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 24;
constexpr int64_t kMaxW4K = (int64_t)1 << 20;
constexpr int64_t kMaxStride = ((int64_t)1 << 31) - 1;

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
    if (ldx < K || ldx % 8 != 0 || ldx > kMaxStride || ldb < K / 2 || ldb % 16 != 0 || ldb > kMaxStride ||
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

qlin_status launch(const w4::Args &a, int64_t experts, void *stream)
{
    if (a.M > 65535 * 128)
        return QLIN_ERR_BAD_SHAPE;
    const int group = a.K / a.G;
    static const w4::Launch kStream[3] = {w4::launch_stream_32, w4::launch_stream_64, w4::launch_stream_128};
    static const w4::Launch kTile[3] = {w4::launch_tile_32, w4::launch_tile_64, w4::launch_tile_128};
    const w4::Launch fn = (a.M <= w4::kStreamTokens ? kStream : kTile)[group == 128 ? 2 : group == 64 ? 1 : 0];
    return fn(a, (int)experts, static_cast<hipStream_t>(stream)) == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

qlin_status qlin_w4_mm(int64_t M, int64_t N, int64_t K, int64_t group, const uint16_t *X,
                       int64_t ldx, const uint8_t *B, int64_t ldb, qlin_scale_type st,
                       const void *b_scale, const uint8_t *b_zero, uint16_t *Y, int64_t ldy,
                       void *stream)
{
    const qlin_status r = check(M, N, K, group, X, ldx, B, ldb, st, b_scale, Y, ldy);
    if (r != QLIN_OK || M == 0 || N == 0)
        return r;
    return launch(make_args(M, N, K, group, X, ldx, B, ldb, st, b_scale, b_zero, Y, ldy), 1, stream);
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
    return launch(a, groups, stream);
}

}  // extern "C"
