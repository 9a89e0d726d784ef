// Products with 4-bit weights: what the kernels and the dispatcher share.
//
//   Y[m,n] = bf16( sum_g s[n,g] * sum_{k in g} X[m,k] * (q[n,k] - z[n,g]) )
//
// Codes become bf16 without a conversion: bf16 holds 7 mantissa bits, so the
// bit pattern 0x4300 | q is the number 128 + q exactly.  The matrix cores then
// sum x * (128 + q) over a group in fp32, and
//   sum x (q - z) = sum x (128 + q) - (128 + z) * sum x
// takes the rest away, the sum of x over the group being one for all weight
// rows.  Products are exact; what the larger terms cost is fp32 rounding of
// sums up to 136/8 times as large, 2^-20 relative beside the 2^-8 of the
// result's rounding to bf16.
//
// Where a row of X is not finite, or so large that 143 x overflows fp32, that
// difference is NaN although the formula's value may not be: such outputs are
// computed again from the formula in fp64 (exact_value), a wave for each.
#pragma once

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qlin_device.h"
#include "qlin_dpp.h"
#include "qlin_moe_scan.h"
#include "qlin_w4_plan.h"
#include "qlinear.h"

namespace qlin {
namespace w4 {

struct Args {
    const uint16_t *x;
    const uint8_t *b;
    const uint8_t *scale;
    const uint8_t *zero;          // or NULL: 8
    uint16_t *y;
    const int32_t *group_off;     // experts' row offsets, or NULL
    int64_t b_gstride;            // bytes between experts' weights
    int64_t ldx, ldb, ldy;        // elements, bytes, elements
    int M;                        // rows (experts: the bound on an expert's rows)
    int rows;                     // experts: rows of X and Y
    int experts;                  // 0 without experts
    int N, K, G;                  // G = K / group
    int st;                       // qlin_scale_type
    int tb, rb;                   // tile kernel: the tile,
    int tiles;                    // token tiles of the grid
    int splits;                   // parts of K, summed by a second kernel
    int split_k;                  // codes of a part
    float *part;                  // [splits][M][N] sums of the parts
};

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// The first row m0 of the workgroup's tile `y` among those; narrows the
// arguments to its expert, whose rows are held inside the buffers whatever the
// offsets say.  Counting the experts' tiles here, 64 experts at a time, keeps
// the grid near the work: a grid of max_rows for every expert would be mostly
// workgroups that leave at once (32 tokens, 128 experts: 49152, of which 9 in
// 10).  False: no such tile.
template <int TILE>
__device__ inline bool enter_tile(Args &a, int y, int &m0)
{
    if (!a.group_off) {
        m0 = y * TILE;
        return m0 < a.M;
    }
    // (offsets of the next 64 are on their way meanwhile; past the last expert the
    // last offset twice, which is no rows)
    const int lane = threadIdx.x & 63;
    int from = a.group_off[min(lane, a.experts)], to = a.group_off[min(lane + 1, a.experts)];
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
        int beg;
        const int rows = expert_rows(from, to, a.rows, a.M, beg);
        from = a.group_off[min(e0 + 64 + lane, a.experts)];
        to = a.group_off[min(e0 + 65 + lane, a.experts)];
        const int tiles = (rows + TILE - 1) / TILE, scan = wave_scan(tiles);
        const int all = __builtin_amdgcn_readlane(scan, 63);
        if (y < all) {
            const int at = __builtin_ctzll(__ballot(scan > y));
            beg = __builtin_amdgcn_readlane(beg, at);
            a.M = __builtin_amdgcn_readlane(rows, at);
            m0 = (y - __builtin_amdgcn_readlane(scan - tiles, at)) * TILE;
            a.x += (int64_t)beg * a.ldx;
            a.y += (int64_t)beg * a.ldy;
            a.b += (e0 + at) * a.b_gstride;
            const int64_t sb = (int64_t)(e0 + at) * a.N * a.G;
            a.scale += sb * (a.st == QLIN_SCALE_F32 ? 4 : 2);
            if (a.zero)
                a.zero += sb;
            return true;
        }
        y -= all;
    }
    return false;
}

// Eight codes of one dword -> 128 + q as eight bf16, the nibbles four apart
// side by side: 0 4 1 5 2 6 3 7.  Seven instructions; the natural order takes
// nine.  `magic` holds 0x4300 twice in a vector register, which the compiler
// is not told: an instruction takes one constant, and that is the mask.
__device__ inline uint32_t expand_magic(uint32_t v)
{
    asm volatile("" : "+v"(v));
    return v;
}

__device__ inline v4i expand8(uint32_t w, uint32_t magic)
{
    const uint32_t mask = 0x000f000fu;
    v4i r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = (int)(((w >> (4 * i)) & mask) | magic);
    }
    return r;
}

// The same in the order of k, for operands that are copied into LDS as they
// are: nibbles become bytes, `up` (a byte for each, at most 15) is added to
// them four at a time, and a byte permutation puts pairs beside the upper
// bytes of 128: nine instructions, eleven with `up`.  `magic` holds 0x43 four
// times.  (Nibble pairs shifted 16 bits apart, the rest added to each of the
// four results: ten and fourteen.)
template <bool UP>
__device__ inline v4i expand8_natural(uint32_t w, uint32_t magic, uint32_t up)
{
    uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
    if (UP) {
        even += up;
        odd += up;
    }
    const uint32_t low = __builtin_amdgcn_perm(odd, even, 0x05010400u);
    const uint32_t high = __builtin_amdgcn_perm(odd, even, 0x07030602u);
    return v4i{(int)__builtin_amdgcn_perm(low, magic, 0x00050004u), (int)__builtin_amdgcn_perm(low, magic, 0x00070006u),
               (int)__builtin_amdgcn_perm(high, magic, 0x00050004u),
               (int)__builtin_amdgcn_perm(high, magic, 0x00070006u)};
}

// Eight tokens' values in the order of expand8.
__device__ inline v4i operand_order(v4i x)
{
    v4i r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r[2 * i] = (int)__builtin_amdgcn_perm((uint32_t)x[2 + i], (uint32_t)x[i], 0x05040100u);
        r[2 * i + 1] = (int)__builtin_amdgcn_perm((uint32_t)x[2 + i], (uint32_t)x[i], 0x07060302u);
    }
    return r;
}

__device__ inline v4f mma(v4i a, v4i b, v4f c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c,
                                                   0, 0, 0);
}

// All of the wave's loads and LDS copies have arrived (vmcnt 0), in a form
// that the compiler counts too: its own waits would otherwise still expect
// the loads before it, and wait for copies issued since.
__device__ inline void wait_loads()
{
    __builtin_amdgcn_s_waitcnt(0x0f70);
    asm volatile("" ::: "memory");
}

// lds_dma16 from a uniform base and the lane's offset.
__device__ inline void lds_dma16_at(const uint8_t *base, uint32_t offset, const void *lds)
{
    const unsigned to = (unsigned)(size_t)lds;
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(offset), "s"(base), "s"(__builtin_amdgcn_readfirstlane(to))
                 : "memory", "m0");
}

// A scale from its 16 (the rest is anything) or 32 bits.
template <int SB>
__device__ inline float scale_value(uint32_t bits, int st)
{
    if (SB == 4)
        return __uint_as_float(bits);
    const float h = __half2float(__ushort_as_half((uint16_t)bits));
    return st == QLIN_SCALE_BF16 ? __uint_as_float(bits << 16) : h;
}

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

// Eight lanes load a row's 128-byte line, lane l (of 64) its 16 bytes
// line_piece(l); lane (n, q) finds the 16 bytes 4 (n / 8) + q of row n mod 8 in
// lane from_line(n, q).  The upper 32 lanes have their pieces in pairs the other
// way round (still 64 bytes for four lanes in a row): half a wave then asks 32
// different banks, not each of 16 twice.
__device__ inline int line_piece(int lane) { return (lane & 7) ^ ((lane >> 4) & 2); }
__device__ inline int from_line(int n, int q) { return 8 * (n & 7) + ((4 * (n >> 3) + q) ^ ((n >> 1) & 2)); }

// The same for half lines, four lanes each: 16 bytes q of row n.
__device__ inline int half_piece(int lane) { return (lane & 3) ^ ((lane >> 4) & 2); }
__device__ inline int from_half(int n, int q) { return 4 * n + (q ^ ((n >> 2) & 2)); }

// Two 16-byte loads of whole 128-byte lines, rows 0..7 and 8..15 of a block:
// lane (n, q) of a load has row n mod 8 and the 16 bytes q of the line's
// first half (n < 8) or second half (n >= 8).  Afterwards `a` holds the first
// half and `b` the second, lane (n, q) the 16 bytes q of row n.
__device__ inline void halves(v4i &a, v4i &b)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int x = a[i], y = b[i];
        // row_ror:8; banks 2 and 3 are lanes 8..15 of each 16
        a[i] = __builtin_amdgcn_update_dpp(x, y, 0x128, 0xF, 0xC, false);
        b[i] = __builtin_amdgcn_update_dpp(y, x, 0x128, 0xF, 0x3, false);
    }
}

// A wave's 16-byte load brings lane (n, quarter q) the codes k = 32 q .. 32 q
// + 31 of row n of a 128-code step: four dwords, one matrix instruction each,
// an instruction summing over the four quarters.  With groups of 128 that is
// one group.  With shorter groups the dwords change quarters first, so that
// an instruction's four quarters hold one group (of 64: two instructions).
// quarters(): that exchange; k_of(j, q): the k at which the eight codes of
// instruction j in quarter q then start.
template <int GROUP>
__device__ inline void quarters(v4i &w)
{
    if (GROUP == 128)
        return;
    const v2u a = __builtin_amdgcn_permlane32_swap((uint32_t)w[0], (uint32_t)w[2], false, false);
    const v2u b = __builtin_amdgcn_permlane32_swap((uint32_t)w[1], (uint32_t)w[3], false, false);
    if (GROUP == 64) {
        w = v4i{(int)a[0], (int)b[0], (int)a[1], (int)b[1]};
    } else {
        const v2u c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
        const v2u d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
        w = v4i{(int)c[0], (int)c[1], (int)d[0], (int)d[1]};
    }
}

template <int GROUP>
__device__ inline int k_of(int j, int q)
{
    return GROUP == 128 ? 32 * q + 8 * j
         : GROUP == 64  ? 32 * (2 * (j >> 1) + (q & 1)) + 8 * ((j & 1) + 2 * (q >> 1))
                        : 32 * j + 8 * q;
}

// The formula's value in fp64, for an output whose fast value is not finite.  The
// whole wave computes it, all lanes with the same m and n: a lane takes 32 codes
// at a time, the lanes of a group add theirs, one of them scales the group's sum.
// A row that has one costs its N walks over K: 1000 tokens with an infinity each
// on 10240 x 5120 18 ms (one of them 0.28 ms, none 0.14 ms), one of 32 on 5120 x
// 25600 3.6 ms.  (A lane by itself over all of K: 107, 1.5 and 15 ms.)
__device__ inline float exact_value(const Args &a, int64_t m, int64_t n)
{
    const int lane = threadIdx.x & 63, chunks = a.K / 32, per = chunks / a.G;
    const uint8_t *b = a.b + n * a.ldb;
    const uint8_t *x = reinterpret_cast<const uint8_t *>(a.x + m * a.ldx);
    double sum = 0.0;
    for (int c0 = 0; c0 < chunks; c0 += 64) {
        const int c = min(c0 + lane, chunks - 1);
        const int64_t at = n * a.G + c / per;
        const float s = a.st == QLIN_SCALE_F32
                            ? reinterpret_cast<const float *>(a.scale)[at]
                            : scale_value<2>(reinterpret_cast<const uint16_t *>(a.scale)[at], a.st);
        const int z = a.zero ? a.zero[at] & 15 : 8;
        double part = 0.0;
#pragma unroll 1                                    // (registers: the callers' occupancy)
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(b + 16 * (int64_t)c + 4 * i);
            const v4i xs = ld16(x + 64 * (int64_t)c + 16 * i);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int q = (w >> (4 * k)) & 15;
                const uint32_t pair = (uint32_t)xs[k / 2];
                part = fma((double)(q - z), (double)__uint_as_float(k & 1 ? pair & 0xffff0000u : pair << 16), part);
            }
        }
        if (per > 1)
            part += dpp_partner(part, 0);
        if (per > 2)
            part += dpp_partner(part, 1);
        if (c0 + lane < chunks && lane % per == 0)
            sum = fma((double)s, part, sum);
        if (__ballot(part != part || sum != sum))
            return __uint_as_float(0x7fc00000u);        // nothing brings it back
    }
    return (float)wave_sum(sum);
}

__device__ inline bool is_finite(float v) { return fabsf(v) <= 3.4028234663852886e38f; }

// v, or the exact value of output (m, n) where `again` holds, one lane's after
// another: every lane of the wave calls.
__device__ inline float recompute(const Args &a, bool again, int m, int n, float v)
{
    for (uint64_t left = __ballot(again); left; left &= left - 1) {
        const int l = __builtin_ctzll(left);
        const float e = exact_value(a, __builtin_amdgcn_readlane(m, l), __builtin_amdgcn_readlane(n, l));
        if ((int)(threadIdx.x & 63) == l)
            v = e;
    }
    return v;
}

// The output of a lane that has one (`there`): rounded to bf16, or computed again
// where it is not finite.  Every lane of the wave calls.
__device__ inline void store_value(const Args &a, bool there, int m, int n, float v)
{
    v = recompute(a, there && !is_finite(v), m, n, v);
    if (there)
        a.y[m * a.ldy + n] = bf16_bits(v);
}

// Launchers, one unit per group length; hipErrorInvalidConfiguration, and nothing
// launched, where the grid would have more threads.
typedef hipError_t (*Launch)(const Args &a, hipStream_t s);
hipError_t launch_stream_32(const Args &a, hipStream_t s);
hipError_t launch_stream_64(const Args &a, hipStream_t s);
hipError_t launch_stream_128(const Args &a, hipStream_t s);
hipError_t launch_tile_32(const Args &a, hipStream_t s);
hipError_t launch_tile_64(const Args &a, hipStream_t s);
hipError_t launch_tile_128(const Args &a, hipStream_t s);

}  // namespace w4
}  // namespace qlin
