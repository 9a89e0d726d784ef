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
// (of 8 weight rows, or of 8 tokens; bytes in the order of line_piece), and one
// scale load covers 32 rows x the slot's two halves.  Afterwards lane (n, q)
// takes the 16 bytes q of row n mod 8's first half line for n < 8, of its second
// for n >= 8.  Columns 0..7 of a product are then 8 rows over
// the slot's first 128 codes, columns 8..15 the same rows over the other 128,
// and the token operand has the 8 tokens' first 128 values in rows 0..7 and
// the other 128 in rows 8..15.  The two diagonal 8 x 8 blocks are wanted, the
// other two are not looked at.
//
// A wave keeps one slot in flight, its codes, scales and token operands all in
// registers, and four or five waves on a SIMD hide each other's waits.  (Two slots
// take 160 to 210 registers, two or three waves: with groups of 128 the same time
// on 51200 x 5120, with groups of 32 and for experts, most of whose workgroups have
// nothing to do, 10 to 35% more; 27 tokens, top-8, 64 experts of 809 x 1216 23.0
// against 18.0 us then, 14.0 now.)  The waves' sums meet in LDS and are added in wave order: no
// second launch, no workspace, and the same bits every time.
//
// The bytes bound it from below and the vector instructions come close behind:
// 226 for 256 codes of 32 rows, half of which turn codes into bf16, keep the
// vector units busy for 40% of the counted cycles, a third of which are the launch's
// start and end.  One token on 51200 x 5120: 30 us, 4.5 TB/s; 32 tokens through 128
// experts of 1536 x 2048: 35 to 43 us by the experts hit.
#pragma once

#include "qlin_w4.h"

namespace qlin {
namespace w4 {

// Where a lane's loads go: bases of the workgroup's rows at code 0, and the
// lane's offsets from them (bytes; of scales, elements).
template <int U>
struct Lane {
    const uint8_t *wbase, *xbase, *sbase, *zbase;
    uint32_t w[U], x, s[(U + 3) / 4], z[(U + 3) / 4];
};

// A slot's codes, scales, zero points and token operands, as loaded.  WHOLE: K
// has 256 codes at least, and a slot that would pass its end is the last 256.
template <int U, int GROUP, int SB, bool ZERO, int ENDS>
struct Slot {
    static constexpr bool WHOLE = ENDS != kShort;
    static constexpr int NG = 128 / GROUP;          // groups of a half
    static constexpr int SW = (NG * SB + 3) / 4;    // dwords of their scales
    static constexpr int SL = (U + 3) / 4;          // scale loads: 32 rows each
    v4i w[U], x[4];
    uint32_t s[SL][SW], z[SL];

    // Addresses are a uniform base and the lane's 32-bit offset from it: rows
    // of the workgroup lie less than 2^31 bytes apart.
    __device__ inline void load(const Args &a, const Lane<U> &o, int k0, int lane)
    {
        if (WHOLE) {
            k0 = min(k0, a.K - kSlot);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = ld16(o.xbase + 2 * k0 + 64 * j + o.x);
            // (where rows are not whole lines, a line's other part is the next
            // slot's or row's and worth keeping: 8 tokens on 40875 x 6272 41.8
            // and so 39.0 us)
#pragma unroll
            for (int u = 0; u < U; ++u)
                w[u] = ENDS == kWhole ? ld_nt(o.wbase + k0 / 2 + o.w[u]) : ld16(o.wbase + k0 / 2 + o.w[u]);
            // Whole dwords, where a lane's own would be less, both halves' or
            // more: a narrower load's value is widened in an operation of its
            // own, which the compiler puts, with its wait, right behind it.
            const int g0 = k0 / GROUP, gz = ZERO && NG == 1 ? min(g0, a.G - 4) : g0;
#pragma unroll
            for (int l = 0; l < SL; ++l) {
                __builtin_memcpy(s[l], o.sbase + (int64_t)SB * g0 + o.s[l] * SB, SB * (NG * SB == 2 ? 2 : NG));
                if (ZERO)
                    __builtin_memcpy(&z[l], o.zbase + gz + o.z[l], 4);
            }
            return;
        }
        // past the end of K the tokens are made zeros and any codes do
        const int seg = line_piece(lane);
        const int over = max(k0 + 32 * seg - (a.K - 32), 0);
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = ld_nt(o.wbase + (k0 - over) / 2 + o.w[u]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + 128 * (seg >> 2) + 32 * j + 8 * (seg & 3);
            x[j] = ld16(o.xbase + 2 * (k0 + 32 * j - max(k - (a.K - 8), 0)) + o.x);
        }
        const int g0 = k0 / GROUP + (lane & 1) * NG;
#pragma unroll
        for (int l = 0; l < SL; ++l) {
            z[l] = 0;
#pragma unroll
            for (int i = 0; i < SW; ++i) s[l][i] = 0;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int64_t at = min(g0 + i, a.G - 1) + (int64_t)o.z[l];
                if (SB == 4)
                    s[l][i] = reinterpret_cast<const uint32_t *>(o.sbase)[at];
                else
                    s[l][i / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(o.sbase)[at] << (16 * (i & 1));
                if (ZERO)
                    z[l] |= (uint32_t)o.zbase[at] << (8 * i);
            }
        }
    }

    // Uses of the slot come after this point of the program: the compiler
    // moves an operation on a scale up to the slot before otherwise, and its
    // wait with it.
    __device__ inline void arrive()
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(x[j]));
#pragma unroll
        for (int u = 0; u < U; ++u) asm volatile("" : "+v"(w[u]));
#pragma unroll
        for (int l = 0; l < SL; ++l) {
#pragma unroll
            for (int i = 0; i < SW; ++i) asm volatile("" : "+v"(s[l][i]));
            if (ZERO)
                asm volatile("" : "+v"(z[l]));
        }
    }
};

// total += the slot's products.
// An instruction takes 32 codes in a row, which keeps the token loads in whole
// pieces of 64 bytes, whatever the group.
template <int U, int GROUP, int SB, bool ZERO, int ENDS>
__device__ inline void add_slot(v4f *total, Slot<U, GROUP, SB, ZERO, ENDS> &slot, int k0, const Args &a,
                                int lane, uint32_t magic)
{
    constexpr bool WHOLE = ENDS != kShort;
    typedef Slot<U, GROUP, SB, ZERO, ENDS> S;
    constexpr int PER = GROUP / 32;                 // matrix instructions of a group
    const v4i ones = {0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80};
    const int n = lane & 15, q = lane >> 4;
    const int from = from_line(n, q), from_s = 2 * (n & 7) + (n >> 3);
    slot.arrive();
    v4i x[4], w[U];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = from_lane(from, slot.x[j]);
        if (!WHOLE && k0 + 128 * (n >> 3) + 32 * j + 8 * q >= a.K)
            x[j] = zero4i();
        x[j] = operand_order(x[j]);
    }
    const int at = ENDS == kInside ? min(k0, a.K - kSlot) : k0;
    if (ENDS == kInside && at < k0) {
        // K ends inside the slot, which holds its last 256 codes: the slot
        // before has had these values already
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at + 128 * (n >> 3) + 32 * j + 8 * q < k0)
                x[j] = zero4i();
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
        if (!ZERO)
            sum_x[g] *= -136.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        // (what the loads took of the other half is shifted out)
        const int half = n >> 3;
        uint32_t s[S::SW], z = 0;
#pragma unroll
        for (int i = 0; i < S::SW; ++i) s[i] = from_lane(from_s + 16 * (u & 3), slot.s[u / 4][i]);
        if (WHOLE && S::NG * SB == 2)
            s[0] >>= 16 * half;
        if (ZERO) {
            z = from_lane(from_s + 16 * (u & 3), slot.z[u / 4]);
            if (WHOLE && S::NG < 4)
                z >>= 8 * (S::NG * half + (S::NG == 1 ? max(at / GROUP - (a.G - 4), 0) : 0));
        }
#pragma unroll
        for (int g = 0; g < 4 / PER; ++g) {
            v4f acc = sum_x[g];                     // what the codes are too large by, times x
            if (ZERO)
                acc *= -128.0f - (float)((z >> (8 * g)) & 15u);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                acc = mma(x[g * PER + i], expand8((uint32_t)w[u][g * PER + i], magic), acc);
            const float sv = scale_value<SB>(SB == 4 ? s[g] : S::NG == 1 ? s[0] : s[g / 2] >> (16 * (g & 1)), a.st);
#pragma unroll
            for (int i = 0; i < 4; ++i) total[u][i] = fmaf(sv, acc[i], total[u][i]);
        }
    }
}

template <int U, int GROUP, int SB, bool ZERO, int ENDS>
__global__ void __launch_bounds__(64 * kStreamWaves) k_stream(Args a)
{
    constexpr bool WHOLE = ENDS != kShort;
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
    Lane<U> o;
    o.wbase = a.b + (int64_t)n0 * a.ldb;
    o.xbase = reinterpret_cast<const uint8_t *>(a.x + (int64_t)m0 * a.ldx);
    o.sbase = a.scale + (int64_t)n0 * a.G * SB;
    o.zbase = ZERO ? a.zero + (int64_t)n0 * a.G : nullptr;
    // rows past the end repeat the last; absent tokens' compute what nobody reads
    o.x = (uint32_t)min(lane >> 3, tokens - 1) * (uint32_t)(2 * a.ldx) + 256 * ((lane >> 2) & 1) + 16 * (line_piece(lane) & 3);
#pragma unroll
    for (int u = 0; u < U; ++u)
        o.w[u] = (uint32_t)min(8 * u + (lane >> 3), a.N - 1 - n0) * (uint32_t)a.ldb + 16 * line_piece(lane);
#pragma unroll
    for (int l = 0; l < SL; ++l) {
        o.z[l] = (uint32_t)min(32 * l + min(lane >> 1, 8 * U - 1), a.N - 1 - n0) * (uint32_t)a.G;
        o.s[l] = o.z[l] + (WHOLE && 128 / GROUP * SB != 2 ? (lane & 1) * (128 / GROUP) : 0);
        if (WHOLE && GROUP == 32)
            o.z[l] += (lane & 1) * 4;
    }
    v4f total[U];
#pragma unroll
    for (int u = 0; u < U; ++u) total[u] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    const uint32_t magic = expand_magic(0x43004300u);
    const int stride = waves * kSlot;
    Slot<U, GROUP, SB, ZERO, ENDS> slot;
    slot.load(a, o, wave * kSlot, lane);
    for (int k0 = wave * kSlot; k0 < a.K; k0 += stride) {
        __builtin_amdgcn_sched_barrier(0);
        add_slot<U, GROUP, SB, ZERO, ENDS>(total, slot, k0, a, lane, magic);
        // unconditional, so that waits stay counted: past the end of K it
        // reads the row's last line again
        slot.load(a, o, k0 + stride, lane);
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
    for (int e = threadIdx.x; e - lane < tokens * 8 * U; e += blockDim.x) {     // whole waves: see store_value
        const int col = e % (8 * U), tok = e / (8 * U);               // rows fastest: stores side by side
        const bool there = tok < tokens && n0 + col < a.N;
        float v = 0.0f;
        if (there)
            for (int w = 0; w < 2 * waves; ++w) v += part[(w * U + (col >> 3)) * 64 + tok * 8 + (col & 7)];
        store_value(a, there, m0 + tok, n0 + col, v);
    }
}

template <int U, int GROUP, int SB, bool ZERO, int ENDS>
hipError_t launch_stream_as(const Args &a, int waves, hipStream_t s)
{
    const int64_t grid = (int64_t)((a.N + 8 * U - 1) / (8 * U)) * row_tiles(a.M, a.experts, a.rows, kStreamTokens);
    waves = min(waves, (a.K + kSlot - 1) / kSlot);
    if (grid * 64 * waves > kMostThreads)
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_stream<U, GROUP, SB, ZERO, ENDS>), dim3((unsigned)grid), dim3(64 * waves),
                       waves * U * 512, s, a);
    return hipGetLastError();
}

template <int GROUP, int SB, bool ZERO, int ENDS>
hipError_t stream_pick(const Args &a, hipStream_t s)
{
    const StreamPick p = pick_stream(a.N, a.K, a.experts, a.rows);
    switch (p.u) {
    case 1: return launch_stream_as<1, GROUP, SB, ZERO, ENDS>(a, p.waves, s);
    case 2: return launch_stream_as<2, GROUP, SB, ZERO, ENDS>(a, p.waves, s);
    default: return launch_stream_as<4, GROUP, SB, ZERO, ENDS>(a, p.waves, s);
    }
}

template <int GROUP, int SB, bool ZERO>
hipError_t stream_ends(const Args &a, hipStream_t s)
{
    switch (stream_end(a.K, a.G)) {
    case kWhole: return stream_pick<GROUP, SB, ZERO, kWhole>(a, s);
    case kInside: return stream_pick<GROUP, SB, ZERO, kInside>(a, s);
    default: return stream_pick<GROUP, SB, ZERO, kShort>(a, s);
    }
}

template <int GROUP>
hipError_t stream_any(const Args &a, hipStream_t s)
{
    if (a.st == QLIN_SCALE_F32)
        return a.zero ? stream_ends<GROUP, 4, true>(a, s) : stream_ends<GROUP, 4, false>(a, s);
    return a.zero ? stream_ends<GROUP, 2, true>(a, s) : stream_ends<GROUP, 2, false>(a, s);
}

}  // namespace w4
}  // namespace qlin
