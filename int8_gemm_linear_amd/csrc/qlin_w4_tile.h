// 4-bit products of more than 8 tokens: tiles on the matrix cores.
//
// A workgroup of four waves owns 16 TB tokens and 64 RB weight rows, 16 RB a
// wave.  The tokens of KS codes at a time are copied straight into LDS, two
// stages ahead through three buffers, in the order in which the matrix
// instructions take their operands; each wave loads its own rows' codes and
// scales into registers, one stage ahead, and expands them there, once for
// all tokens.  A group's products are summed by themselves, starting from
// what its sum of x takes away, then scaled and added to the totals.  That
// sum of x is the same for all weight rows: a stage ahead, each wave computes
// it for some of the tokens with products by ones and leaves it in LDS.
//
// Where M x N is too few tiles for the 256 CUs, K is split over workgroups
// whose sums a second kernel adds in order.
//
// With many tokens the vector units, which expand codes and scale sums, are busy for
// 47% and the matrix cores for 40% of the time: a wave expands a group before its
// products and scales after them, and the two or three waves of a SIMD overlap that
// in part only.  1000 tokens on 10240 x 5120 134 us, 780 TFLOP/s; 2048 tokens 232 us,
// 925 TFLOP/s.  With few, it is the time of a stage, from its loads to its products,
// over the parts of K: 32 tokens on 5120 x 25600 with zero points 34 us.  16 000 rows
// of 128 experts on 2048 x 768 109 us, 460 TFLOP/s: six stages a tile, which starting
// and ending it outweigh.
#pragma once

#include "qlin_w4.h"

namespace qlin {
namespace w4 {

constexpr int kTileWaves = 4;

// Where a lane's loads go: bytes from the wave's first row (of scales: elements).
template <int RB, int H>
struct Lane {
    const uint8_t *wbase, *sbase, *zbase;
    uint32_t w[RB][H], s;
};

// The codes, scales and zero points of a wave's rows for a stage, as loaded:
// in an order that is good for the cache (the L1 takes one access for each 64
// bytes that four lanes in a row ask for together), which a permutation of the
// lanes turns into the matrix operands'.  Eight lanes load a row where a stage
// has whole 128-byte lines (KS = 256, two loads for 16 rows), four where it has
// half lines, and lane l the scales of row l.
// (1000 tokens on 10240 x 5120: 167 us, with loads in the operands' order 171.)
template <int RB, int KS, int GROUP, int SB, bool ZERO, bool WHOLE>
struct Codes {
    static constexpr int H = KS / 128, NG = KS / GROUP;
    v4i w[RB][H];
    uint32_t s[(SB * NG + 3) / 4], z[(NG + 3) / 4];

    // Addresses are a uniform base, the wave's first row at code 0, and the
    // lane's 32-bit offset from it.
    __device__ inline void load(const Args &a, const Lane<RB, H> &o, int k0, int lane)
    {
        if (WHOLE) {
            k0 = min(k0, a.K - KS);
            const int64_t g0 = k0 / GROUP;
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int h = 0; h < H; ++h) w[r][h] = ld16(o.wbase + k0 / 2 + o.w[r][h]);
            __builtin_memcpy(s, o.sbase + SB * g0 + SB * o.s, SB * NG);
            if (ZERO)
                __builtin_memcpy(z, o.zbase + g0 + o.s, NG);
            return;
        }
        // past the end of K the tokens are zeros and any codes do
        const int over = max(k0 + 32 * (H == 2 ? line_piece(lane) : half_piece(lane)) - (a.K - 32), 0);
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int h = 0; h < H; ++h) w[r][h] = ld16(o.wbase + (k0 - over) / 2 + o.w[r][h]);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int64_t at = min(k0 / GROUP + i, a.G - 1) + (int64_t)o.s;
            __builtin_memcpy(reinterpret_cast<uint8_t *>(s) + SB * i, o.sbase + SB * at, SB);
            if (ZERO)
                reinterpret_cast<uint8_t *>(z)[i] = o.zbase[at];
        }
    }

    // The codes in the operands' order: lane (n, q) the 16 bytes q of row n of
    // each step of 128 codes.
    __device__ inline void permute(int n, int q)
    {
        const int from = H == 2 ? from_line(n, q) : from_half(n, q);
#pragma unroll
        for (int r = 0; r < RB; ++r) {
#pragma unroll
            for (int h = 0; h < H; ++h) w[r][h] = from_lane(from, w[r][h]);
            if (H == 2)
                halves(w[r][0], w[r][H - 1]);
        }
    }

    __device__ inline float scale(int r, int n, int i, int st) const
    {
        const uint32_t v = from_lane(16 * r + n, s[SB == 4 ? i : i / 2]);
        return scale_value<SB>(SB == 4 ? v : v >> (16 * (i & 1)), st);
    }

    // 15 - z in each byte: added to the codes it makes them 143 + (q - z), and
    // what has to be taken away the same for all rows.
    __device__ inline uint32_t raise(int r, int n, int i) const
    {
        const uint32_t zero = (from_lane(16 * r + n, z[i / 4]) >> (8 * (i & 3))) & 15u;
        return (15u - zero) * 0x01010101u;
    }
};

// What a token's pieces are exchanged by.  Together are read (measured, a pair of
// lanes at a time) tokens 0-3 and 12-15 of one quarter of the wave with 4-11 of the
// next, and the others; a quarter's pieces are four places from the next one's, or
// all quarters' the same four.  So the token's upper two bits count down: 0, 3, 2,
// 1 keeps both apart (with the token itself, 0 to 3, each place of one quarter met
// one of the other: half as many again LDS cycles, 1000 tokens on 10240 x 5120
// 148 us, so 138 us).
__device__ inline int mix(int t) { return (4 * (-(t >> 2) & 3)) | (t & 3); }

// A grid of gx weight tiles by `tiles` token tiles, in chunks of one weight tile
// by up to 8 token tiles.  Workgroups go to the 8 XCDs in turn, so id mod 8 names
// the L2: each takes every 8th chunk, so that what runs at once shares both its
// weights and its tokens there (2048 tokens on 10240 x 5120, as it was then: 287 us
// against 305 us with all token tiles of a weight tile in a row); the workgroups of
// the chunks that are left over go to the XCDs one by one (every 8th weight tile to
// an XCD, and none to some where there are fewer than 8: 9660 rows of 16 experts on
// 100 x 1152 47 us, so 19 us; 1000 tokens on 5120 x 25600 536 and 435 us).
struct Blocks {
    int high, blocks;                   // token tiles of a chunk, such blocks
    int64_t all;                        // workgroups of a part of K
};
__host__ __device__ inline Blocks tile_blocks(int gx, int tiles)
{
    const int blocks = (tiles + 7) / 8, high = (tiles + blocks - 1) / blocks;
    return Blocks{high, blocks, ((int64_t)gx * blocks * high + 7) & ~(int64_t)7};
}

template <int TB, int RB, int KS, int GROUP, int SB, bool ZERO, int ENDS>
__global__ void __launch_bounds__(64 * kTileWaves, 2) k_tile(Args a)
{
    constexpr bool WHOLE = ENDS != kShort;
    constexpr int H = KS / 128, PIECES = KS / 8, PER = GROUP / 32, NS = KS / GROUP;
    constexpr int COPIES = 16 * TB * PIECES / 64;           // 1 KB each
    const int gx = (a.N + 64 * RB - 1) / (64 * RB);
    const Blocks bl = tile_blocks(gx, a.tiles);
    const int all = (int)bl.all, split = blockIdx.x / all, id = blockIdx.x % all;
    const int each = gx * bl.blocks / 8 * bl.high;          // an XCD's workgroups of whole chunks
    const int j = id >> 3, rest = 8 * each + (j - each) * 8 + (id & 7);
    const int chunk = j < each ? j / bl.high * 8 + (id & 7) : rest / bl.high;
    const int nx = chunk % gx, y = chunk / gx * bl.high + (j < each ? j : rest) % bl.high;
    int m0;
    if (y >= a.tiles || !enter_tile<16 * TB>(a, y, m0))
        return;
    __shared__ v4i lds[3][16 * TB * PIECES];
    __shared__ v4f sums[2][NS][TB * 4];             // [group][token / 4], times what the codes are too large by
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, q = lane >> 4;
    const int n0 = (nx * kTileWaves + wave) * 16 * RB;
    const int kbeg = split * a.split_k, kend = min(a.K, kbeg + a.split_k);
    // (a wave past the last row repeats it)
    const int first = min(n0, a.N - 1);
    Lane<RB, H> o;
    o.wbase = a.b + (int64_t)first * a.ldb;
    o.sbase = a.scale + (int64_t)first * a.G * SB;
    o.zbase = ZERO ? a.zero + (int64_t)first * a.G : nullptr;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
#pragma unroll
        for (int h = 0; h < H; ++h)
            o.w[r][h] = (uint32_t)min(H == 2 ? 16 * r + 8 * h + (lane >> 3) : 16 * r + (lane >> 2), a.N - 1 - first) *
                            (uint32_t)a.ldb + 16 * (H == 2 ? line_piece(lane) : half_piece(lane));
    }
    o.s = (uint32_t)min(lane & (16 * RB - 1), a.N - 1 - first) * (uint32_t)a.G;
    v4f total[RB][TB];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int t = 0; t < TB; ++t) total[r][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    // Place p of token t holds the values of codes 8 (p xor mix(t)) .. of its
    // step, so that the lanes whose 16 bytes are read at once meet 16 different
    // places of the 256 bytes in which the banks repeat, and four lanes of a copy
    // still read 64 bytes side by side.  A wave's copies are 4 KB apart: the
    // lane's place in them is one.
    const int copy_t = (wave * 64 + lane) / PIECES, copy_p = lane % PIECES;
    const int copy_piece = (copy_p ^ mix(copy_t)) & 15;
    static_assert(256 / PIECES % 16 == 0 || 256 / PIECES == 8, "tokens of a wave's copies");
    // (eight tokens on, bit 3 of the exchange is the other)
    auto piece_at = [&](int i) { return 256 / PIECES == 8 ? copy_piece ^ (8 * (i & 1)) : copy_piece; };
    uint32_t copy_x[COPIES / kTileWaves];                   // bytes from the first token at code 0
#pragma unroll
    for (int i = 0; i < COPIES / kTileWaves; ++i) {
        copy_x[i] = (uint32_t)min(copy_t + i * (256 / PIECES), a.M - 1 - m0) * (uint32_t)(2 * a.ldx) +
                    256 * (copy_p >> 4) + 16 * piece_at(i);
    }
    const uint8_t *xbase = reinterpret_cast<const uint8_t *>(a.x + (int64_t)m0 * a.ldx);
    auto stage = [&](int k0, int buf) {
        if (WHOLE)
            k0 = min(k0, a.K - KS);
#pragma unroll
        for (int i = 0; i < COPIES / kTileWaves; ++i) {
            v4i *to = &lds[buf][(i * kTileWaves + wave) * 64];
            if (WHOLE || k0 + 128 * (copy_p >> 4) + 8 * piece_at(i) < kend)
                lds_dma16_at(xbase + 2 * (int64_t)k0, copy_x[i], to);
            else
                to[lane] = zero4i();
        }
    };
    int place[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) place[j] = n * PIECES + ((k_of<GROUP>(j, q) / 8) ^ mix(n));

    const v4i ones = {0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80};
    auto sum = [&](int buf, int to) {
#pragma unroll
        for (int i = 0; i < (TB * H + kTileWaves - 1) / kTileWaves; ++i) {
            const int task = i * kTileWaves + wave, t = task / H, h = task % H;
            if (task >= TB * H)
                break;
#pragma unroll
            for (int g = 0; g < 4 / PER; ++g) {
                v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < PER; ++j) s = mma(lds[buf][place[g * PER + j] + 16 * h + 16 * t * PIECES], ones, s);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] *= ZERO ? -143.0f : -136.0f;
                if (n == 0)
                    sums[to][h * (4 / PER) + g][t * 4 + q] = s;
            }
        }
    };

    const uint32_t magic = expand_magic(0x43434343u);
    Codes<RB, KS, GROUP, SB, ZERO, WHOLE> cur, next;
    stage(kbeg, 0);
    stage(kbeg + KS, 1);
    cur.load(a, o, kbeg, lane);
    wait_loads();
    __syncthreads();
    sum(0, 0);
    int buf = 0, par = 0;
    for (int k0 = kbeg; k0 < kend; k0 += KS) {
        const int buf1 = buf == 2 ? 0 : buf + 1, buf2 = buf1 == 2 ? 0 : buf1 + 1;
        // the next stage's tokens have landed; this stage's sums are there; the last stage's buffer is free
        wait_loads();
        __syncthreads();
        if (ENDS == kInside && k0 > a.K - KS) {
            // K ends inside the stage, which holds its last KS codes: the
            // tokens' values that the stage before had already are made zeros
#pragma unroll
            for (int i = 0; i < COPIES / kTileWaves; ++i)
                if (a.K - KS + 128 * (copy_p >> 4) + 8 * piece_at(i) < k0)
                    lds[buf][(i * kTileWaves + wave) * 64 + lane] = zero4i();
            __syncthreads();
            sum(buf, par);
            __syncthreads();
        }
        const v4i *xs = lds[buf];
        cur.permute(n, q);
#pragma unroll
        for (int h = 0; h < H; ++h) {
#pragma unroll
            for (int r = 0; r < RB; ++r) quarters<GROUP>(cur.w[r][h]);
#pragma unroll
            for (int g = 0; g < 4 / PER; ++g) {
                const int at = h * (4 / PER) + g;
                v4i b[RB][PER];
                float sv[RB];
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    const uint32_t up = ZERO ? cur.raise(r, n, at) : 0;
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        // expanded here and not earlier, where registers are not free yet
                        uint32_t w = (uint32_t)cur.w[r][h][g * PER + i];
                        asm volatile("" : "+v"(w));
                        b[r][i] = expand8_natural<ZERO>(w, magic, up);
                    }
                    sv[r] = cur.scale(r, n, at, a.st);
                }
                // The products of a token block, while the operands of the
                // next come from LDS (each into the registers of the one just
                // used) and the sums of the last are scaled.
                v4f acc[2][RB], s;
                v4i x[PER];
                auto fetch = [&](int t, int i) { x[i] = xs[place[g * PER + i] + 16 * h + 16 * t * PIECES]; };
                s = sums[par][at][q];
#pragma unroll
                for (int i = 0; i < PER; ++i) fetch(0, i);
                // Where three waves share a SIMD, the one at its products goes
                // before those that expand codes (1000 tokens on 5120 x 8192, groups
                // of 64, 156 and so 151 us; with two waves, 2048 tokens on 10240 x
                // 5120, 241 and so 248 us).
                if (TB * RB < 16)
                    __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int t = 0; t <= TB; ++t) {
                    // What the stage asks of memory, and the next one's sums,
                    // go between its products; always, for a branch would
                    // keep them apart: past the end of K they repeat the last
                    // stage (or read zeros), and nobody looks.
                    if (at == 0 && t == 0)
                        stage(k0 + 2 * KS, buf2);
                    if (at == 0 && t == (TB > 1 ? 1 : 0))
                        next.load(a, o, k0 + KS, lane);
                    if (at == 0 && t == (TB > 2 ? 2 : TB))
                        sum(buf1, par ^ 1);
                    if (t < TB) {
#pragma unroll
                        for (int r = 0; r < RB; ++r)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[t & 1][r][i] = s[i];
                        if (t + 1 < TB)
                            s = sums[par][at][(t + 1) * 4 + q];
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
#pragma unroll
                            for (int r = 0; r < RB; ++r) acc[t & 1][r] = mma(x[i], b[r][i], acc[t & 1][r]);
                            if (t + 1 < TB)
                                fetch(t + 1, i);
                        }
                    }
                    if (t > 0) {
#pragma unroll
                        for (int r = 0; r < RB; ++r)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                total[r][t - 1][i] = fmaf(sv[r], acc[(t - 1) & 1][r][i], total[r][t - 1][i]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (TB * RB < 16)
                    __builtin_amdgcn_s_setprio(0);
            }
        }
        cur = next;
        buf = buf1;
        par ^= 1;
    }

    wait_loads();                                           // the copies past the end have landed
    // lane (n, q) holds tokens 4 q .. 4 q + 3 of row n
    if (a.splits > 1) {
        float *part = a.part + (int64_t)split * a.M * a.N;
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = m0 + 16 * t + 4 * q + i;
#pragma unroll
                for (int r = 0; r < RB; ++r)
                    if (m < a.M && n0 + 16 * r + n < a.N)
                        part[(int64_t)m * a.N + n0 + 16 * r + n] = total[r][t][i];
            }
        return;
    }
    // The wave's values change places in LDS, so that lanes store 16 bytes and
    // 2 RB of them a token's (16 000 rows of 128 experts, N 2048, K 768: 119 us;
    // two bytes each, 16 lanes side by side: 127 us).  Rows are 16 bytes longer than
    // they need to be: the four rows that are written at once are then in
    // different banks.
    constexpr int ROW = 16 * RB + 8;
    static_assert(kTileWaves * 16 * TB * ROW * 2 <= (int)sizeof(lds), "a tile of values");
    __syncthreads();                                        // the last stage's tokens are read
    uint16_t *mine = reinterpret_cast<uint16_t *>(lds) + wave * 16 * TB * ROW;
    bool fine = true;
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                mine[(16 * t + 4 * q + i) * ROW + 16 * r + n] = bf16_bits(total[r][t][i]);
                fine = fine && is_finite(total[r][t][i]);
            }
    if (__ballot(!fine))
        // rare: the lanes look their values over again, in a loop that costs no registers above
        for (int e = 0; e < 4 * TB * RB; ++e) {
            const int t = 16 * (e / (4 * RB)) + 4 * q + e / RB % 4, c = 16 * (e % RB) + n;
            uint16_t &v = mine[t * ROW + c];
            const bool again = m0 + t < a.M && n0 + c < a.N && (v & 0x7f80) == 0x7f80;
            const float f = recompute(a, again, m0 + t, n0 + c, 0.0f);
            if (again)
                v = bf16_bits(f);
        }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    constexpr int PIECES_OUT = 16 * TB * 2 * RB;
#pragma unroll
    for (int i = 0; i < (PIECES_OUT + 63) / 64; ++i) {
        const int u = 64 * i + lane, t = u / (2 * RB), c = 8 * (u % (2 * RB));
        if (u >= PIECES_OUT || m0 + t >= a.M || n0 + c >= a.N)
            continue;
        const uint16_t *from = mine + t * ROW + c;
        uint16_t *to = a.y + (m0 + t) * a.ldy + n0 + c;
        if (n0 + c + 8 <= a.N)
            __builtin_memcpy(to, from, 16);
        else
            for (int k = 0; k < a.N - n0 - c; ++k) to[k] = from[k];
    }
}

template <int TB, int RB, int KS, int GROUP, int SB, bool ZERO, int ENDS>
hipError_t launch_tile_as(Args a, hipStream_t s)
{
    const int64_t tiles = row_tiles(a.M, a.experts, a.rows, 16 * TB);
    if (tiles > 0x7fffffff / 8)
        return hipErrorInvalidConfiguration;
    a.tiles = (int)tiles;
    const Blocks bl = tile_blocks((a.N + 64 * RB - 1) / (64 * RB), a.tiles);
    const int64_t grid = bl.all * a.splits;
    if (grid * 64 * kTileWaves > kMostThreads)
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_tile<TB, RB, KS, GROUP, SB, ZERO, ENDS>), dim3((unsigned)grid), dim3(64 * kTileWaves), 0, s, a);
    return hipGetLastError();
}

template <int TB, int RB, int KS, int GROUP, int SB, bool ZERO>
hipError_t tile_ends(const Args &a, hipStream_t s)
{
    if (tile_end(a.K, KS) == kWhole)
        return launch_tile_as<TB, RB, KS, GROUP, SB, ZERO, kWhole>(a, s);
    return launch_tile_as<TB, RB, KS, GROUP, SB, ZERO, kInside>(a, s);
}

template <int GROUP, int SB, bool ZERO>
hipError_t tile_pick(const Args &a, hipStream_t s)
{
    if (a.K < 128)
        return launch_tile_as<kShortTile.tb, kShortTile.rb, kShortTile.ks, GROUP, SB, ZERO, kShort>(a, s);
    switch (10 * a.tb + a.rb) {
    case 11: return tile_ends<1, 1, 256, GROUP, SB, ZERO>(a, s);
    case 12: return tile_ends<1, 2, 256, GROUP, SB, ZERO>(a, s);
    case 21: return tile_ends<2, 1, 256, GROUP, SB, ZERO>(a, s);
    case 22: return tile_ends<2, 2, 256, GROUP, SB, ZERO>(a, s);
    case 42: return tile_ends<4, 2, 128, GROUP, SB, ZERO>(a, s);
    default: return tile_ends<4, 4, 128, GROUP, SB, ZERO>(a, s);
    }
}

template <int GROUP>
hipError_t tile_any(const Args &a, hipStream_t s)
{
    if (a.st == QLIN_SCALE_F32)
        return a.zero ? tile_pick<GROUP, 4, true>(a, s) : tile_pick<GROUP, 4, false>(a, s);
    return a.zero ? tile_pick<GROUP, 2, true>(a, s) : tile_pick<GROUP, 2, false>(a, s);
}

}  // namespace w4
}  // namespace qlin
