// 4-bit products of up to 8 tokens: the weights are read once, straight into
// registers, and everything else hides behind them.
//
// A workgroup owns 8 U weight rows and all tokens; its waves share K in slots
// of 256 codes (one 128-byte line of each row), slot i going to wave i mod W.
//
// Loads go by the cache, products by the matrix cores, and a permutation of
// the lanes lies between.  The L1 takes one access for each 64 bytes that
// four lanes in a row ask for together, and 64 accesses for lanes that each
// ask elsewhere; with loads in the order of the matrix operands those accesses
// alone took 34 us for 131 MB.  So lane l loads 16 bytes l mod 8 of row l / 8
// (of 8 weight rows, or of 8 tokens), and one scale load covers 32 rows x the
// slot's two halves.  Afterwards lane (n, q) takes from lane 8 (n mod 8) +
// 4 (n / 8) + q: the 16 bytes q of row n mod 8's first half line for n < 8,
// of its second for n >= 8.  Columns 0..7 of a product are then 8 rows over
// the slot's first 128 codes, columns 8..15 the same rows over the other 128,
// and the token operand has the 8 tokens' first 128 values in rows 0..7 and
// the other 128 in rows 8..15.  The two diagonal 8 x 8 blocks are wanted, the
// other two are not looked at.
//
// A wave keeps AHEAD slots in flight, each with its codes, scales and token
// operands, all in registers: loads return in order, so they arrive together
// and nothing waits for more than it needs.  The waves' sums meet in LDS and
// are added in wave order: no second launch, no workspace, and the same bits
// every time.
#pragma once

#include "qlin_w4.h"

namespace qlin {
namespace w4 {

constexpr int kSlot = 256;
constexpr int kStreamWaves = 8;

__device__ inline uint32_t from_lane(int lane, uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_ds_bpermute(4 * lane, (int)v);
}

__device__ inline v4i from_lane(int lane, v4i v)
{
    v4i r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (int)from_lane(lane, (uint32_t)v[i]);
    return r;
}

// A slot's codes, scales, zero points and token operands, as loaded.  EVEN: K
// % 128 == 0.
template <int U, int GROUP, int SB, bool ZERO, bool EVEN>
struct Slot {
    static constexpr int NG = 128 / GROUP;          // groups of a half
    static constexpr int SW = (NG * SB + 3) / 4;    // dwords of their scales
    static constexpr int SL = (U + 3) / 4;          // scale loads: 32 rows each
    v4i w[U], x[4];
    uint32_t s[SL][SW], z[SL];

    __device__ inline void load(const Args &a, const uint8_t *const *wrow, const uint8_t *const *srow,
                                const uint8_t *const *zrow, const uint16_t *xrow, int k0, int lane)
    {
        const int seg = lane & 7;
        // past the end of K the tokens are made zeros and any codes do
        const int at = min(k0 + 32 * seg, a.K - 32) / 2;
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = ld_nt(wrow[u] + at);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = ld16(reinterpret_cast<const uint8_t *>(
                xrow + min(k0 + 128 * (seg >> 2) + 32 * j + 8 * (seg & 3), a.K - 8)));
        const int g0 = min(k0 + 128 * (lane & 1), EVEN ? a.K - 128 : a.K - 32) / GROUP;
#pragma unroll
        for (int l = 0; l < SL; ++l) {
            z[l] = 0;
            s[l][0] = 0;
            if (EVEN) {
                __builtin_memcpy(s[l], srow[l] + SB * g0, NG * SB);
                if (ZERO)
                    __builtin_memcpy(&z[l], zrow[l] + g0, NG);
            } else {
#pragma unroll
                for (int i = 1; i < SW; ++i) s[l][i] = 0;
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    const int g = min(g0 + i, a.G - 1);
                    if (SB == 4)
                        s[l][i] = reinterpret_cast<const uint32_t *>(srow[l])[g];
                    else
                        s[l][i / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(srow[l])[g] << (16 * (i & 1));
                    if (ZERO)
                        z[l] |= (uint32_t)zrow[l][g] << (8 * i);
                }
            }
        }
    }
};

// total += the slot's products; `partial` where the slot passes the end of K.
// An instruction takes 32 codes in a row, which keeps the token loads in whole
// pieces of 64 bytes, whatever the group.
template <int U, int GROUP, int SB, bool ZERO, bool EVEN>
__device__ inline void add_slot(v4f *total, const Slot<U, GROUP, SB, ZERO, EVEN> &slot, int k0, bool partial,
                                const Args &a, int lane, uint32_t magic)
{
    typedef Slot<U, GROUP, SB, ZERO, EVEN> S;
    constexpr int PER = GROUP / 32;                 // matrix instructions of a group
    const v4i ones = {0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80};
    const int n = lane & 15, q = lane >> 4;
    const int from = 8 * (n & 7) + 4 * (n >> 3) + q, from_s = 2 * (n & 7) + (n >> 3);
    v4i x[4], w[U];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = from_lane(from, slot.x[j]);
        if (partial && k0 + 128 * (n >> 3) + 32 * j + 8 * q >= a.K)
            x[j] = zero4i();
        x[j] = operand_order(x[j]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        w[u] = from_lane(from, slot.w[u]);
        quarters<32>(w[u]);
    }
    v4f sum_x[4 / PER];
#pragma unroll
    for (int g = 0; g < 4 / PER; ++g) {
        sum_x[g] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < PER; ++i) sum_x[g] = mma(x[g * PER + i], ones, sum_x[g]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint32_t s[S::SW], z = 0;
#pragma unroll
        for (int i = 0; i < S::SW; ++i) s[i] = from_lane(from_s + 16 * (u & 3), slot.s[u / 4][i]);
        if (ZERO)
            z = from_lane(from_s + 16 * (u & 3), slot.z[u / 4]);
#pragma unroll
        for (int g = 0; g < 4 / PER; ++g) {
            v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < PER; ++i)
                acc = mma(x[g * PER + i], expand8((uint32_t)w[u][g * PER + i], magic), acc);
            const float sv = scale_value<SB>(SB == 4 ? s[g] : S::NG == 1 ? s[0] & 0xffffu
                                                            : (s[g / 2] >> (16 * (g & 1))) & 0xffffu, a.st);
            const float zv = ZERO ? -128.0f - (float)((z >> (8 * g)) & 0xffu) : -136.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) total[u][i] = fmaf(sv, fmaf(zv, sum_x[g][i], acc[i]), total[u][i]);
        }
    }
}

template <int U, int AHEAD, int GROUP, int SB, bool ZERO, bool EVEN>
__global__ void __launch_bounds__(64 * kStreamWaves) k_stream(Args a)
{
    const int gx = (a.N + 8 * U - 1) / (8 * U);
    int m0;
    if (!enter_tile<kStreamTokens>(a, blockIdx.x / gx, m0))
        return;
    extern __shared__ float part[];                 // [wave][half][u][token][row]
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = (int)(blockIdx.x % gx) * 8 * U;
    const int tokens = min(a.M - m0, kStreamTokens);
    constexpr int SL = (U + 3) / 4;
    // the rows of absent tokens compute what nobody reads
    const uint16_t *xrow = a.x + (int64_t)(m0 + min(lane >> 3, tokens - 1)) * a.ldx;
    const uint8_t *wrow[U], *srow[SL], *zrow[SL];
#pragma unroll
    for (int u = 0; u < U; ++u) wrow[u] = a.b + (int64_t)min(n0 + 8 * u + (lane >> 3), a.N - 1) * a.ldb;
#pragma unroll
    for (int l = 0; l < SL; ++l) {
        const int64_t row = min(n0 + 32 * l + min(lane >> 1, 8 * U - 1), a.N - 1);
        srow[l] = a.scale + row * a.G * SB;
        zrow[l] = ZERO ? a.zero + row * a.G : nullptr;
    }
    v4f total[U];
#pragma unroll
    for (int u = 0; u < U; ++u) total[u] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    const uint32_t magic = expand_magic();
    const int stride = waves * kSlot;
    Slot<U, GROUP, SB, ZERO, EVEN> slot[AHEAD];
    int k0 = wave * kSlot;
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) slot[d].load(a, wrow, srow, zrow, xrow, k0 + d * stride, lane);
    __builtin_amdgcn_sched_barrier(0);
    const int left = a.K > k0 ? (a.K - k0 + stride - 1) / stride : 0;          // the wave's slots
    for (int i = 0; i < left / AHEAD; ++i) {
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
            add_slot(total, slot[d], k0, k0 + kSlot > a.K, a, lane, magic);
            // unconditional, so that waits stay counted: past the end of K it
            // reads the row's last line again
            slot[d].load(a, wrow, srow, zrow, xrow, k0 + AHEAD * stride, lane);
            k0 += stride;
            // keeps these loads before the next slot's wait
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int d = 0; d < AHEAD - 1; ++d)
        if (d < left % AHEAD) {
            add_slot(total, slot[d], k0, k0 + kSlot > a.K, a, lane, magic);
            k0 += stride;
        }

    const int n = lane & 15, q = lane >> 4;
    // lane (n, q) holds operand rows 4 q .. 4 q + 3 of column n: wanted where both are of the same half
    if (n >> 3 == q >> 1) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[((wave * 2 + (n >> 3)) * U + u) * 64 + (4 * (q & 1) + i) * 8 + (n & 7)] = total[u][i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < tokens * 8 * U; e += blockDim.x) {
        const int col = e % (8 * U), tok = e / (8 * U);               // rows fastest: stores side by side
        if (n0 + col >= a.N)
            continue;
        float v = 0.0f;
        for (int w = 0; w < 2 * waves; ++w) v += part[(w * U + (col >> 3)) * 64 + tok * 8 + (col & 7)];
        store_value(a, m0 + tok, n0 + col, v);
    }
}

template <int U, int AHEAD, int GROUP, int SB, bool ZERO, bool EVEN>
hipError_t launch_stream_as(const Args &a, int waves, hipStream_t s)
{
    const int64_t grid = (int64_t)((a.N + 8 * U - 1) / (8 * U)) * row_tiles(a, kStreamTokens);
    if (grid > 0x7fffffff)
        return hipErrorInvalidValue;
    waves = min(waves, (a.K + kSlot - 1) / kSlot);
    hipLaunchKernelGGL((k_stream<U, AHEAD, GROUP, SB, ZERO, EVEN>), dim3((unsigned)grid), dim3(64 * waves),
                       waves * U * 512, s, a);
    return hipGetLastError();
}

template <int GROUP, int SB, bool ZERO, bool EVEN>
hipError_t stream_pick(const Args &a, hipStream_t s)
{
    const int64_t rows = (int64_t)a.N * max(a.experts, 1);
    if (rows <= 16 * 256)
        return launch_stream_as<1, 2, GROUP, SB, ZERO, EVEN>(a, 4, s);
    if (a.M <= 2 || rows <= 32 * 1024)
        return launch_stream_as<2, 2, GROUP, SB, ZERO, EVEN>(a, 4, s);
    return launch_stream_as<4, 2, GROUP, SB, ZERO, EVEN>(a, 4, s);
}

template <int GROUP, int SB, bool ZERO>
hipError_t stream_even(const Args &a, hipStream_t s)
{
    // groups of 128 divide K by themselves
    if (GROUP == 128 || a.K % 128 == 0)
        return stream_pick<GROUP, SB, ZERO, true>(a, s);
    return stream_pick<GROUP, SB, ZERO, GROUP == 128>(a, s);
}

template <int GROUP>
hipError_t stream_any(const Args &a, hipStream_t s)
{
    if (a.st == QLIN_SCALE_F32)
        return a.zero ? stream_even<GROUP, 4, true>(a, s) : stream_even<GROUP, 4, false>(a, s);
    return a.zero ? stream_even<GROUP, 2, true>(a, s) : stream_even<GROUP, 2, false>(a, s);
}

}  // namespace w4
}  // namespace qlin
