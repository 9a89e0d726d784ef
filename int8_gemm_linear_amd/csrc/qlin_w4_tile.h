// 4-bit products of more than 8 tokens: tiles on the matrix cores.
//
// A workgroup owns 16 TB tokens and 16 RB W weight rows, W waves side by side
// along the rows.  The tokens of KS codes at a time are copied straight into
// LDS (two buffers) in the order in which the matrix instructions take their
// operands; each wave loads its own rows' codes and scales into registers,
// one stage ahead, and expands them there, once for all tokens.  A group's
// products are summed by themselves, corrected by its sum of x, scaled and
// added to the totals in registers.
#pragma once

#include "qlin_w4.h"

namespace qlin {
namespace w4 {

// The codes, scales and zero points of a wave's rows for a stage.  With KS =
// 256 two loads take whole 128-byte lines of 8 rows each (see halves()).
template <int RB, int KS, int GROUP, int SB, bool ZERO>
struct Codes {
    static constexpr int H = KS / 128, NG = KS / GROUP;
    v4i w[RB][H];
    uint32_t s[RB][NG], z[RB][NG];

    __device__ inline void load(const Args &a, const uint8_t *const (*wrow)[H], const uint8_t *const *srow,
                                const uint8_t *const *zrow, int k0, int n, int q)
    {
        // past the end of K the tokens are zeros and any codes do
        const int at = min(k0 + 32 * q + (H == 2 ? 128 * (n >> 3) : 0), a.K - 32) / 2;
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int h = 0; h < H; ++h) w[r][h] = ld16(wrow[r][h] + at);
        const int g0 = k0 / GROUP;
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int g = min(g0 + i, a.G - 1);
                s[r][i] = SB == 4 ? reinterpret_cast<const uint32_t *>(srow[r])[g]
                                  : reinterpret_cast<const uint16_t *>(srow[r])[g];
                z[r][i] = ZERO ? zrow[r][g] : 8;
            }
    }
};

template <int TB, int RB, int KS, int GROUP, int SB, bool ZERO>
__global__ void __launch_bounds__(256) k_tile(Args a)
{
    constexpr int H = KS / 128, PIECES = KS / 8, PER = GROUP / 32;
    if (!enter_expert(a))
        return;
    __shared__ v4i lds[2][16 * TB * PIECES];
    const int m0 = blockIdx.y * 16 * TB;
    if (m0 >= a.M)
        return;
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, q = lane >> 4;
    const int n0 = (blockIdx.x * waves + wave) * 16 * RB;
    const uint8_t *wrow[RB][H], *srow[RB], *zrow[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        const int base = n0 + 16 * r;
#pragma unroll
        for (int h = 0; h < H; ++h)
            wrow[r][h] = a.b + (int64_t)min(H == 2 ? base + 8 * h + (n & 7) : base + n, a.N - 1) * a.ldb;
        const int64_t row = min(base + n, a.N - 1);
        srow[r] = a.scale + row * a.G * SB;
        zrow[r] = ZERO ? a.zero + row * a.G : nullptr;
    }
    v4f total[RB][TB];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int t = 0; t < TB; ++t) total[r][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    // place p of token t holds the step's piece p with its bits 2 and 3
    // exchanged by t: a read of 16 tokens x 4 pieces meets every bank equally
    auto stage = [&](int k0, int buf) {
        for (int i = wave; i < 16 * TB * PIECES / 64; i += waves) {
            const int at = i * 64 + lane, t = at / PIECES, p = at % PIECES;
            const int k = k0 + 128 * (p >> 4) + k_of<GROUP>(((p >> 2) & 3) ^ (t & 3), p & 3);
            if (k < a.K)
                lds_dma16(a.x + (int64_t)min(m0 + t, a.M - 1) * a.ldx + k, &lds[buf][i * 64]);
            else
                lds[buf][at] = zero4i();
        }
    };
    int place[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) place[j] = n * PIECES + 4 * (j ^ (n & 3)) + q;

    const uint32_t magic = expand_magic();
    const v4i ones = {0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80};
    Codes<RB, KS, GROUP, SB, ZERO> cur, next;
    stage(0, 0);
    cur.load(a, wrow, srow, zrow, 0, n, q);
    for (int k0 = 0, buf = 0; k0 < a.K; k0 += KS, buf ^= 1) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (k0 + KS < a.K) {
            stage(k0 + KS, buf ^ 1);
            next.load(a, wrow, srow, zrow, k0 + KS, n, q);
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            if (H == 2 && h == 0) {
#pragma unroll
                for (int r = 0; r < RB; ++r) halves(cur.w[r][0], cur.w[r][1]);
            }
#pragma unroll
            for (int r = 0; r < RB; ++r) quarters<GROUP>(cur.w[r][h]);
#pragma unroll
            for (int g = 0; g < 4 / PER; ++g) {
                v4i b[RB][PER];
                float sv[RB], zv[RB];
#pragma unroll
                for (int r = 0; r < RB; ++r) {
#pragma unroll
                    for (int i = 0; i < PER; ++i) b[r][i] = expand8_natural((uint32_t)cur.w[r][h][g * PER + i], magic);
                    sv[r] = scale_value<SB>(cur.s[r][h * (4 / PER) + g], a.st);
                    zv[r] = ZERO ? -128.0f - (float)cur.z[r][h * (4 / PER) + g] : -136.0f;
                }
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    v4i x[PER];
                    v4f sum_x = {0.0f, 0.0f, 0.0f, 0.0f}, acc[RB];
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        x[i] = lds[buf][place[g * PER + i] + 16 * h + 16 * t * PIECES];
                        sum_x = mma(x[i], ones, sum_x);
                    }
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        acc[r] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int i = 0; i < PER; ++i) acc[r] = mma(x[i], b[r][i], acc[r]);
                    }
#pragma unroll
                    for (int r = 0; r < RB; ++r)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            total[r][t][i] = fmaf(sv[r], fmaf(zv[r], sum_x[i], acc[r][i]), total[r][t][i]);
                }
            }
        }
        cur = next;
    }

    // lane (n, q) holds tokens 4 q .. 4 q + 3 of row n
    bool fine = true;
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = m0 + 16 * t + 4 * q + i;
            if (m >= a.M)
                continue;
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                if (n0 + 16 * r + n < a.N)
                    a.y[m * a.ldy + n0 + 16 * r + n] = bf16_bits(total[r][t][i]);
                fine = fine && is_finite(total[r][t][i]);
            }
        }
    if (fine)
        return;
    // rare: the lane looks its outputs over again, in a loop that costs no registers above
    for (int e = 0; e < 4 * TB * RB; ++e) {
        const int64_t m = m0 + 16 * (e / (4 * RB)) + 4 * q + e / RB % 4, c = n0 + 16 * (e % RB) + n;
        if (m < a.M && c < a.N && (a.y[m * a.ldy + c] & 0x7f80) == 0x7f80)
            a.y[m * a.ldy + c] = bf16_bits(exact_value(a, m, c));
    }
}

template <int TB, int RB, int KS, int GROUP, int SB, bool ZERO>
hipError_t launch_tile_as(const Args &a, int experts, hipStream_t s)
{
    constexpr int W = 4;
    const dim3 grid((a.N + 16 * RB * W - 1) / (16 * RB * W), (a.M + 16 * TB - 1) / (16 * TB), experts);
    hipLaunchKernelGGL((k_tile<TB, RB, KS, GROUP, SB, ZERO>), grid, dim3(64 * W), 0, s, a);
    return hipGetLastError();
}

template <int GROUP, int SB, bool ZERO>
hipError_t tile_pick(const Args &a, int experts, hipStream_t s)
{
    if (a.M <= 16)
        return launch_tile_as<1, 1, 256, GROUP, SB, ZERO>(a, experts, s);
    if (a.M <= 32)
        return launch_tile_as<2, 1, 256, GROUP, SB, ZERO>(a, experts, s);
    if (a.M <= 64)
        return launch_tile_as<4, 2, 256, GROUP, SB, ZERO>(a, experts, s);
    return launch_tile_as<8, 4, 128, GROUP, SB, ZERO>(a, experts, s);
}

template <int GROUP>
hipError_t tile_any(const Args &a, int experts, hipStream_t s)
{
    if (a.st == QLIN_SCALE_F32)
        return a.zero ? tile_pick<GROUP, 4, true>(a, experts, s) : tile_pick<GROUP, 4, false>(a, experts, s);
    return a.zero ? tile_pick<GROUP, 2, true>(a, experts, s) : tile_pick<GROUP, 2, false>(a, experts, s);
}

}  // namespace w4
}  // namespace qlin
