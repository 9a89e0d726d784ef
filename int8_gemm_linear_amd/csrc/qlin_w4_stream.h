// 4-bit products of up to 8 tokens: the weights are read once, straight into
// registers, and everything else hides behind them.
//
// A workgroup owns 8 U weight rows and all tokens; its waves share K in slots
// of 256 codes (one 128-byte line of each row), slot i going to wave i mod W,
// so that the workgroup reads whole row segments.  A load takes the whole
// lines of 8 rows, 16 bytes a lane (reading half lines of 16 rows instead
// costs a quarter of the bandwidth: 131 MB in 28 us against 21 us), and feeds
// the matrix cores as it comes: lane (n, q) holds the 16 bytes q of row n mod
// 8's first half line for n < 8, of its second for n >= 8.  So columns 0..7
// of a product are 8 rows over the slot's first 128 codes, columns 8..15 the
// same rows over the other 128; the token operand has the 8 tokens' first
// 128 values in rows 0..7 and the other 128 in rows 8..15.  The two diagonal
// 8 x 8 blocks are wanted, the other two are not looked at.
//
// A wave keeps the codes and scales of AHEAD slots in flight and nothing
// else: loads return in order, so a load of tokens issued between them would
// wait for all of them.  The tokens come from LDS, where the workgroup puts
// them, in the order of the matrix instructions' operands, for as much of K
// as fits at once.  The waves' sums meet in LDS and are added in wave order:
// no second launch, no workspace, and the same bits every time.
#pragma once

#include "qlin_w4.h"

namespace qlin {
namespace w4 {

constexpr int kSlot = 256;
constexpr int kStreamWaves = 8;
constexpr int kStreamLds = 64 * 1024;       // tokens in LDS at once: two workgroups of a CU

// The codes, scales and zero points of a slot.  EVEN: K % 128 == 0.
template <int U, int GROUP, int SB, bool ZERO, bool EVEN>
struct Slot {
    static constexpr int NG = 128 / GROUP;          // a lane's groups
    static constexpr int SW = (NG * SB + 3) / 4;    // dwords of its scales
    v4i w[U];
    uint32_t s[U][SW];
    uint32_t z[U];

    // k0: the lane's first code (its row's half line)
    __device__ inline void load(const Args &a, const uint8_t *const *wrow, const uint8_t *const *srow,
                                const uint8_t *const *zrow, int k0, int q)
    {
        // past the end of K the tokens are zeros and any codes do
        const int at = min(k0 + 32 * q, a.K - 32) / 2;
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = ld_nt(wrow[u] + at);
        const int g0 = min(k0, EVEN ? a.K - 128 : a.K - 32) / GROUP;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (NG == 1) {
                s[u][0] = SB == 4 ? reinterpret_cast<const uint32_t *>(srow[u])[g0]
                                  : reinterpret_cast<const uint16_t *>(srow[u])[g0];
                z[u] = ZERO ? zrow[u][g0] : 0;
            } else if (EVEN) {
                __builtin_memcpy(s[u], srow[u] + SB * g0, NG * SB);
                z[u] = 0;
                if (ZERO)
                    __builtin_memcpy(&z[u], zrow[u] + g0, NG);
            } else {
#pragma unroll
                for (int i = 0; i < SW; ++i) s[u][i] = 0;
                z[u] = 0;
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    const int g = min(g0 + i, a.G - 1);
                    if (SB == 4)
                        s[u][i] = reinterpret_cast<const uint32_t *>(srow[u])[g];
                    else
                        s[u][i / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(srow[u])[g] << (16 * (i & 1));
                    if (ZERO)
                        z[u] |= (uint32_t)zrow[u][g] << (8 * i);
                }
            }
        }
    }

    __device__ inline float scale(int u, int i, int st) const
    {
        return scale_value<SB>(SB == 4 ? s[u][i] : NG == 1 ? s[u][0] : (s[u][i / 2] >> (16 * (i & 1))) & 0xffffu, st);
    }

    // -(128 + z)
    __device__ inline float bias(int u, int i) const
    {
        return ZERO ? -128.0f - (float)((z[u] >> (8 * i)) & 0xffu) : -136.0f;
    }
};

// 16-byte pieces from one token's values of k codes to the next's: one more
// than they take, so that the 8 tokens that read one piece meet different
// banks.
__host__ __device__ inline int token_pitch(int k) { return k / 8 + 1; }

// Tokens' values of codes c0 .. to LDS, in operand order: piece 4 j + q of a
// step of 128 holds k_of(j, q).  T x P loads of a thread are in flight at
// once: a load from L2 takes as long as one of the weights.
template <int GROUP, int T, int P>
__device__ inline void stage_tokens(v4i *lds, int pitch, const uint16_t *x, int64_t ldx, int tokens, int c0, int K,
                                    int pieces)
{
    for (int p0 = threadIdx.x; p0 < pieces; p0 += P * blockDim.x) {
        v4i v[P][T];
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const int k = c0 + 8 * (p0 + i * (int)blockDim.x);
                v[i][t] = ld16(reinterpret_cast<const uint8_t *>(x + min(t, tokens - 1) * ldx + min(k, K - 8)));
            }
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const int p = p0 + i * (int)blockDim.x;
                if (t < tokens && p < pieces)
                    lds[t * pitch + (p & ~15) + piece_of<GROUP>(p)] = c0 + 8 * p < K ? operand_order(v[i][t]) : zero4i();
            }
    }
}

// total += the slot's products with the tokens; x: the lane's token pieces.
template <int U, int GROUP, typename S>
__device__ inline void add_slot(v4f *total, S &slot, const v4i *x, int st, uint32_t magic)
{
    constexpr int PER = GROUP / 32;                 // matrix instructions of a group
    const v4i ones = {0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80};
#pragma unroll
    for (int u = 0; u < U; ++u) quarters<GROUP>(slot.w[u]);
#pragma unroll
    for (int g = 0; g < 4 / PER; ++g) {
        v4i xv[PER];
        v4f sum_x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            xv[i] = x[4 * (g * PER + i)];
            sum_x = mma(xv[i], ones, sum_x);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < PER; ++i) acc = mma(xv[i], expand8((uint32_t)slot.w[u][g * PER + i], magic), acc);
            const float sv = slot.scale(u, g, st), zv = slot.bias(u, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) total[u][i] = fmaf(sv, fmaf(zv, sum_x[i], acc[i]), total[u][i]);
        }
    }
}

template <int U, int AHEAD, int GROUP, int SB, bool ZERO, bool EVEN>
__global__ void __launch_bounds__(64 * kStreamWaves) k_stream(Args a, int kc)
{
    const int gx = (a.N + 8 * U - 1) / (8 * U);
    int m0;
    if (!enter_tile<kStreamTokens>(a, blockIdx.x / gx, m0))
        return;
    extern __shared__ v4i lds[];
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, q = lane >> 4;
    const int n0 = (int)(blockIdx.x % gx) * 8 * U;
    const int tokens = min(a.M - m0, kStreamTokens);
    const int pitch = token_pitch(min(kc, (a.K + kSlot - 1) / kSlot * kSlot));
    const uint8_t *wrow[U], *srow[U], *zrow[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = min(n0 + 8 * u + (n & 7), a.N - 1);
        wrow[u] = a.b + row * a.ldb;
        srow[u] = a.scale + row * a.G * SB;
        zrow[u] = ZERO ? a.zero + row * a.G : nullptr;
    }
    v4f total[U];
#pragma unroll
    for (int u = 0; u < U; ++u) total[u] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    const uint32_t magic = expand_magic();
    const int stride = waves * kSlot, half = 128 * (n >> 3);
    Slot<U, GROUP, SB, ZERO, EVEN> slot[AHEAD];
    int k0 = wave * kSlot;
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) slot[d].load(a, wrow, srow, zrow, k0 + d * stride + half, q);

    // operand row n: token n mod 8, the slot's half n / 8; the rows of absent tokens compute what nobody reads
    const v4i *mine = lds + min(n & 7, tokens - 1) * pitch + (half >> 3) + q;
    for (int c0 = 0; c0 < a.K; c0 += kc) {          // kc: a multiple of AHEAD * stride
        __syncthreads();
        // piece 4 j + q of a step of 128 holds k_of(j, q)
        const int pieces = (min(kc, a.K - c0) + kSlot - 1) / kSlot * (kSlot / 8);
        if (tokens <= 2)
            stage_tokens<GROUP, 2, 4>(lds, pitch, a.x + (int64_t)m0 * a.ldx, a.ldx, tokens, c0, a.K, pieces);
        else
            stage_tokens<GROUP, 8, 1>(lds, pitch, a.x + (int64_t)m0 * a.ldx, a.ldx, tokens, c0, a.K, pieces);
        __syncthreads();
        const int end = min(c0 + kc, a.K);
        const int left = end > k0 ? (end - k0 + stride - 1) / stride : 0;      // the wave's slots of the chunk
        for (int i = 0; i < left / AHEAD; ++i) {
#pragma unroll
            for (int d = 0; d < AHEAD; ++d) {
                add_slot<U, GROUP>(total, slot[d], mine + (k0 - c0) / 8, a.st, magic);
                // unconditional, so that waits stay counted: past the end of K
                // it reads the row's last line again
                slot[d].load(a, wrow, srow, zrow, k0 + AHEAD * stride + half, q);
                k0 += stride;
                // keeps these loads before the next slot's wait
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // a remainder only where K ends
#pragma unroll
        for (int d = 0; d < AHEAD - 1; ++d)
            if (d < left % AHEAD) {
                add_slot<U, GROUP>(total, slot[d], mine + (k0 - c0) / 8, a.st, magic);
                k0 += stride;
            }
    }

    // lane (n, q) holds operand rows 4 q .. 4 q + 3 of column n: wanted where both are of the same half
    __syncthreads();
    float *part = reinterpret_cast<float *>(lds);           // [wave][half][u][token][row]
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
hipError_t launch_stream_as(const Args &a, int waves, int lds_bytes, hipStream_t s)
{
    const int64_t grid = (int64_t)((a.N + 8 * U - 1) / (8 * U)) * row_tiles(a, kStreamTokens);
    if (grid > 0x7fffffff)
        return hipErrorInvalidValue;
    const int slots = (a.K + kSlot - 1) / kSlot;
    const int tokens = min(a.M, kStreamTokens);
    const int fits = (lds_bytes / (16 * tokens) - 1) * 8;               // codes of K whose tokens fit
    waves = min(waves, min(slots, fits / (AHEAD * kSlot)));
    const int round = AHEAD * waves * kSlot;
    const int kc = min(fits / round, (a.K + round - 1) / round) * round;
    const int lds = max(16 * tokens * token_pitch(min(kc, slots * kSlot)), waves * U * 512);
    hipLaunchKernelGGL((k_stream<U, AHEAD, GROUP, SB, ZERO, EVEN>), dim3((unsigned)grid), dim3(64 * waves), lds,
                       s, a, kc);
    return hipGetLastError();
}

template <int GROUP, int SB, bool ZERO, bool EVEN>
hipError_t stream_pick(const Args &a, hipStream_t s)
{
    const int64_t rows = (int64_t)a.N * max(a.experts, 1);
    if (rows <= 16 * 256)
        return launch_stream_as<1, 2, GROUP, SB, ZERO, EVEN>(a, 4, kStreamLds, s);
    if (a.M <= 2 || rows <= 32 * 1024)
        return launch_stream_as<2, 2, GROUP, SB, ZERO, EVEN>(a, 4, kStreamLds, s);
    return launch_stream_as<4, 2, GROUP, SB, ZERO, EVEN>(a, 4, kStreamLds, s);
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
