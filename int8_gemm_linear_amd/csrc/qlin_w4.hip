// Products with 4-bit weights and group scales:
//   Y[m,n] = bf16( sum_g s[n,g] * sum_{k in g} X[m,k] * (q[n,k] - z[n,g]) ).
//
// One wave per output row n and up to 8 tokens: the lanes share the row's
// bytes 4 at a time (8 codes of one group), multiply in fp32 and scale each
// 8-code sum, and the wave adds its lanes at the end.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qlin_device.h"
#include "qlin_dpp.h"
#include "qlinear.h"

namespace qlin {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 24;
constexpr int64_t kMaxW4K = (int64_t)1 << 20;
constexpr int64_t kMaxStride = ((int64_t)1 << 31) - 1;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

struct W4Args {
    const uint16_t *x;
    const uint8_t *b;
    const void *scale;
    const uint8_t *zero;          // or NULL: 8
    uint16_t *y;
    const int32_t *group_off;     // experts' row offsets, or NULL
    int64_t b_gstride;            // bytes between experts' weights
    int64_t ldx, ldb, ldy;        // elements, bytes, elements
    int M;                        // rows (experts: the bound on an expert's rows)
    int rows;                     // experts: rows of X and Y
    int N, K, G;                  // G = K / group
    int group_log;                // log2 of the group
    int st;                       // qlin_scale_type
};

__device__ inline float load_scale(const void *p, int st, int64_t i)
{
    if (st == QLIN_SCALE_F32)
        return static_cast<const float *>(p)[i];
    const uint16_t h = static_cast<const uint16_t *>(p)[i];
    return st == QLIN_SCALE_BF16 ? __uint_as_float((uint32_t)h << 16)
                                 : __half2float(__ushort_as_half(h));
}

// Narrows the arguments to the workgroup's expert (grid.z); false: no rows.
__device__ inline bool enter_expert(W4Args &a)
{
    if (!a.group_off)
        return true;
    const int e = blockIdx.z;
    const int beg = min(max(a.group_off[e], 0), a.rows), end = min(a.group_off[e + 1], a.rows);
    a.M = min(end - beg, a.M);
    if (a.M <= 0)
        return false;
    a.x += (int64_t)beg * a.ldx;
    a.y += (int64_t)beg * a.ldy;
    a.b += e * a.b_gstride;
    const int64_t sb = (int64_t)e * a.N * a.G;
    a.scale = static_cast<const uint8_t *>(a.scale) + sb * (a.st == QLIN_SCALE_F32 ? 4 : 2);
    if (a.zero)
        a.zero += sb;
    return true;
}

__global__ void __launch_bounds__(256) k_w4(W4Args a)
{
    if (!enter_expert(a))
        return;
    const int lane = threadIdx.x & 63;
    const int n = blockIdx.x * 4 + (threadIdx.x >> 6);
    const int m0 = blockIdx.y * 8;
    if (n >= a.N || m0 >= a.M)
        return;
    float sum[8] = {};
    const int64_t so = (int64_t)n * a.G;
    for (int k = lane * 8; k < a.K; k += 512) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(a.b + (int64_t)n * a.ldb + k / 2);
        const float s = load_scale(a.scale, a.st, so + (k >> a.group_log));
        const int z = a.zero ? a.zero[so + (k >> a.group_log)] : 8;
        float v[8];
        for (int i = 0; i < 8; ++i) v[i] = (float)((int)((w >> (4 * i)) & 15) - z);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            if (m0 + t < a.M) {
                const v4i xv = *reinterpret_cast<const v4i *>(a.x + (int64_t)(m0 + t) * a.ldx + k);
                float p = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t h = (uint32_t)xv[i >> 1];
                    p = fmaf(__uint_as_float(i & 1 ? h & 0xffff0000u : h << 16), v[i], p);
                }
                sum[t] = fmaf(s, p, sum[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const float v = wave_sum(sum[t]);
        if (lane == 0 && m0 + t < a.M)
            a.y[(int64_t)(m0 + t) * a.ldy + n] = bf16_bits(v);
    }
}

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

W4Args make_args(int64_t M, int64_t N, int64_t K, int64_t group, const uint16_t *X, int64_t ldx,
                 const uint8_t *B, int64_t ldb, qlin_scale_type st, const void *scale,
                 const uint8_t *zero, uint16_t *Y, int64_t ldy)
{
    W4Args a{};
    a.x = X;
    a.b = B;
    a.scale = scale;
    a.zero = zero;
    a.y = Y;
    a.ldx = ldx;
    a.ldb = ldb;
    a.ldy = ldy;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.G = (int)(K / group);
    a.group_log = group == 32 ? 5 : group == 64 ? 6 : 7;
    a.st = (int)st;
    return a;
}

qlin_status launch(const W4Args &a, int64_t experts, void *stream)
{
    const int64_t gx = (a.N + 3) / 4, gy = (a.M + 7) / 8;
    if (gy > 65535)
        return QLIN_ERR_BAD_SHAPE;
    hipLaunchKernelGGL(k_w4, dim3((unsigned)gx, (unsigned)gy, (unsigned)experts), dim3(256), 0,
                       static_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
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
    W4Args a = make_args(M, N, K, group, X, ldx, B, ldb, st, b_scale, b_zero, Y, ldy);
    a.group_off = group_offsets;
    a.b_gstride = b_group_stride;
    a.rows = (int)rows;
    return launch(a, groups, stream);
}

}  // extern "C"
