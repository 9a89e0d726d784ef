// Low-rank adapters of many requests beside a shared projection, and their gradients.
//
// Token t has the adapter i = ids[t] (none where that is no adapter), and
//   v[t,r] = sum_k x[t,k] A[i,r,k],        y[t,n] = base[t,n] + s_i sum_r v[t,r] B[i,n,r]
//   u[t,r] = sum_n dy[t,n] B[i,n,r],       dx[t,k] = base[t,k] + s_i sum_r u[t,r] A[i,r,k]
//   dA[i,r,k] = s_i sum_{t of i} u[t,r] x[t,k],   dB[i,n,r] = s_i sum_{t of i} dy[t,n] v[t,r]
//
// Tokens are put in order by adapter first (the plan); a tile is up to 16 TB tokens of
// one adapter.  Three kernels do the products on the bf16 matrix cores:
//   shrink   a long K against few ranks: v, or u from B transposed
//   expand   few ranks against a long N: y, or dx from A transposed
//   outer    sums over an adapter's tokens: dA and dB
// v and u stay fp32 between them.  A matrix core takes them as bf16 pieces: the upper 16
// bits (cut, so that nothing overflows), then the rest.  Two pieces hold 16 bits of the
// mantissa, far below the final rounding to bf16 of y and dx; dA and dB, which are fp32,
// take three, which is all of it.
#include <algorithm>

#include "qlin_device.h"
#include "qlin_moe_scan.h"
#include "qlinear.h"

namespace qlin {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kMaxAdapters = 2048;
constexpr int kMaxRank = 128;
constexpr int64_t kMaxTokens = (int64_t)1 << 24;
constexpr int64_t kMaxWidth = (int64_t)1 << 20;
constexpr int64_t kMaxStride = (int64_t)1 << 31;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

__device__ inline v4f mma(v4i a, v4i b, v4f c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Eight bf16 values at any element's address, of which `n` exist; the others are 0.
__device__ inline v4i load8(const uint16_t *p)
{
    v4i v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

__device__ inline v4i load8(const uint16_t *p, int n)
{
    if (n >= 8)
        return load8(p);
    uint16_t t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = i < n ? p[i] : 0;
    v4i v;
    __builtin_memcpy(&v, t, 16);
    return v;
}

// The upper 16 bits of v as a float, and what is left of it (an infinity leaves nothing).
__device__ inline float cut(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }
__device__ inline float rest(float v, float c) { return fabsf(c) < INFINITY ? v - c : 0.0f; }

__device__ inline int pack2(float lo, float hi)
{
    return (int)((uint32_t)bf16_bits(lo) | (uint32_t)bf16_bits(hi) << 16);
}

// ---------------------------------------------------------------------------
// Plan: tokens by adapter, and the tiles of each.
// ---------------------------------------------------------------------------
constexpr int kPlanWaves = 16, kPlanThreads = 64 * kPlanWaves;
constexpr int kBins = kMaxAdapters + 1;        // the last one in use: tokens without an adapter

struct Plan {
    const void *ids;
    int32_t *order;            // [tokens]: the tokens by (adapter, token); those without one come last
    int32_t *offsets;          // [adapters + 1]: the first place of each adapter
    int4 *tiles;               // [max_tiles]: adapter (-1: none), first place, tokens (0: no tile)
    int tokens, adapters, tile, max_tiles, id_bits;
};

__device__ inline int bin_of(const Plan &p, int t)
{
    const int64_t id = p.id_bits == 64 ? static_cast<const int64_t *>(p.ids)[t] : static_cast<const int32_t *>(p.ids)[t];
    return id >= 0 && id < p.adapters ? (int)id : p.adapters;
}

// One workgroup: a stable counting sort whose waves own contiguous parts of the tokens.
__global__ void __launch_bounds__(kPlanThreads) k_plan(Plan p)
{
    __shared__ int32_t hist[kPlanWaves][kBins];
    __shared__ int32_t sums[2][kPlanWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, bins = p.adapters + 1;
    const int part = (p.tokens + kPlanThreads - 1) / kPlanThreads * 64;
    const int beg = min(wave * part, p.tokens), end = min(beg + part, p.tokens);
    for (int w = 0; w < kPlanWaves; ++w)
        for (int b = tid; b < bins; b += kPlanThreads) hist[w][b] = 0;
    __syncthreads();
    for (int t = beg + lane; t < end; t += 64) atomicAdd(&hist[wave][bin_of(p, t)], 1);
    __syncthreads();
    // a thread takes `each` consecutive adapters: their tokens and tiles before it
    const int each = (bins + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(tid * each, bins), b1 = min(b0 + each, bins);
    int tokens = 0, tiles = 0;
    for (int b = b0; b < b1; ++b) {
        int n = 0;
        for (int w = 0; w < kPlanWaves; ++w) n += hist[w][b];
        tokens += n;
        tiles += (n + p.tile - 1) / p.tile;
    }
    const int scan0 = wave_scan(tokens), scan1 = wave_scan(tiles);
    if (lane == 63) {
        sums[0][wave] = scan0;
        sums[1][wave] = scan1;
    }
    __syncthreads();
    int at = scan0 - tokens, tile = scan1 - tiles, all = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
        at += w < wave ? sums[0][w] : 0;
        tile += w < wave ? sums[1][w] : 0;
        all += sums[1][w];
    }
    for (int b = b0; b < b1; ++b) {
        const int first = at;
        for (int w = 0; w < kPlanWaves; ++w) {
            const int c = hist[w][b];
            hist[w][b] = at;
            at += c;
        }
        p.offsets[b] = first;                  // (that of the last bin: tokens with an adapter)
        for (int t = first; t < at; t += p.tile)
            p.tiles[tile++] = make_int4(b < p.adapters ? b : -1, t, min(p.tile, at - t), 0);
    }
    for (int t = all + tid; t < p.max_tiles; t += kPlanThreads) p.tiles[t] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    int bits = 0;
    while ((1 << bits) < bins) ++bits;
    for (int t = beg; t < end; t += 64) {
        const bool there = t + lane < end;
        const int b = there ? bin_of(p, t + lane) : 0;
        uint64_t same = __ballot(there);
        same = there ? same : ~same;
        for (int i = 0; i < bits; ++i) {
            const uint64_t set = __ballot((b >> i) & 1);
            same &= (b >> i) & 1 ? set : ~set;
        }
        const int lead = __ffsll((unsigned long long)same) - 1;
        int to = 0;
        if (there && lane == lead)
            to = atomicAdd(&hist[wave][b], __popcll(same));
        to = __shfl(to, lead);
        if (there)
            p.order[to + __popcll(same & (((uint64_t)1 << lane) - 1))] = t + lane;
    }
}

// ---------------------------------------------------------------------------
// Shrink: part[split][place][r] = sum over the split's k of x[token,k] w[adapter,r,k].
// Sixteen ranks by sixteen tokens a matrix product; waves share K in steps of 128.
// ---------------------------------------------------------------------------
constexpr int kStep = 128;

struct ShrinkArgs {
    const uint16_t *x, *w;     // w [adapters][R][ldw]
    const int32_t *order;
    const int4 *tiles;
    float *part;               // [splits][tokens][16 RB]
    int64_t ldx, ldw;
    int tokens, K, R, splits;
};

template <int TB, int RB>
__global__ void __launch_bounds__(kThreads) k_shrink(ShrinkArgs a)
{
    __shared__ v4f sums[kWaves - 1][TB * RB][64];
    const int4 tile = a.tiles[blockIdx.x / a.splits];
    const int split = blockIdx.x % a.splits;
    if (tile.x < 0 || tile.z == 0)
        return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    const uint16_t *px[TB], *pw[RB];
#pragma unroll
    for (int t = 0; t < TB; ++t) px[t] = a.x + a.order[tile.y + min(16 * t + i, tile.z - 1)] * a.ldx + 8 * q;
    // (ranks behind R take the last one's row: their sums are not read)
#pragma unroll
    for (int r = 0; r < RB; ++r) pw[r] = a.w + ((int64_t)tile.x * a.R + min(16 * r + i, a.R - 1)) * a.ldw + 8 * q;
    v4f acc[TB][RB] = {};
    const int steps = (a.K + kStep - 1) / kStep, per = (steps + a.splits - 1) / a.splits;
    const int end = min((split + 1) * per, steps);
    for (int s = split * per + wave; s < end; s += kWaves) {
        const int k = s * kStep;
        v4i x[TB][4], w[RB][4];
        if (k + kStep <= a.K) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int t = 0; t < TB; ++t) x[t][j] = load8(px[t] + k + 32 * j);
#pragma unroll
                for (int r = 0; r < RB; ++r) w[r][j] = load8(pw[r] + k + 32 * j);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int left = a.K - (k + 32 * j + 8 * q);
#pragma unroll
                for (int t = 0; t < TB; ++t) x[t][j] = load8(px[t] + k + 32 * j, left);
#pragma unroll
                for (int r = 0; r < RB; ++r) w[r][j] = load8(pw[r] + k + 32 * j, left);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int t = 0; t < TB; ++t)
#pragma unroll
                for (int r = 0; r < RB; ++r) acc[t][r] = mma(x[t][j], w[r][j], acc[t][r]);
    }
    if (wave > 0)
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int r = 0; r < RB; ++r) sums[wave - 1][t * RB + r][lane] = acc[t][r];
    __syncthreads();
    if (wave > 0)
        return;
    float *part = a.part + ((int64_t)split * a.tokens + tile.y) * (16 * RB);
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            v4f v = acc[t][r];
            for (int w = 0; w < kWaves - 1; ++w) v += sums[w][t * RB + r][lane];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (16 * t + 4 * q + c < tile.z)
                    part[(16 * t + 4 * q + c) * (16 * RB) + 16 * r + i] = v[c];
        }
}

// ---------------------------------------------------------------------------
// Expand: out[token,n] = bf16(base[token,n] + s sum_r v[place,r] w[adapter,n,r]).
// A wave takes 64 n at a time as four products of 16; a product's row 4 a + c is
// n = 16 a + 4 j + c, so that a lane ends with 16 n in a row of its token.
// ---------------------------------------------------------------------------
struct ExpandArgs {
    const float *part, *scale;
    const int32_t *order;
    const int4 *tiles;
    const uint16_t *w, *base;  // w [adapters][N][R]
    uint16_t *out;
    int64_t ldb, ldo;
    int tokens, N, R, Rp, splits, chunks;
};

// Ranks 8 c .. 8 c + 7 of a place: the splits' sums in order, times s.
__device__ inline void load_ranks(float (&v)[8], const ExpandArgs &a, int place, int c, float s)
{
    const float *p = a.part + (int64_t)place * a.Rp + 8 * c;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    for (int k = 0; k < a.splits; ++k, p += (int64_t)a.tokens * a.Rp) {
        const v4f lo = *reinterpret_cast<const v4f *>(p), hi = *reinterpret_cast<const v4f *>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] += lo[i];
            v[4 + i] += hi[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s;
}

// G groups of 32 ranks; PACK: at most 16 ranks, both pieces of v in one product.
template <int TB, int G, bool PACK>
__global__ void __launch_bounds__(kThreads) k_expand(ExpandArgs a)
{
    const int4 tile = a.tiles[blockIdx.x / a.chunks];
    const int chunk = blockIdx.x % a.chunks;
    if (tile.z == 0)
        return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    const int ranks = a.R / 8;                 // chunks of 8 ranks
    const bool live = tile.x >= 0;
    int64_t token[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) token[t] = a.order[tile.y + min(16 * t + i, tile.z - 1)];
    v4i hi[TB][G], lo[TB][PACK ? 1 : G];
    const uint16_t *w = a.w + (int64_t)(live ? tile.x : 0) * a.N * a.R;
    if (live) {
        const float s = a.scale ? a.scale[tile.x] : 1.0f;
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int c = PACK ? q % ranks : 4 * g + q, piece = PACK ? q / ranks : 0;
                float v[8] = {}, h[8], l[8];
                if (c < ranks && piece < 2)
                    load_ranks(v, a, tile.y + min(16 * t + i, tile.z - 1), c, s);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    h[e] = cut(v[e]);
                    l[e] = rest(v[e], h[e]);
                    if (PACK && piece == 1)
                        h[e] = l[e];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    hi[t][g][e] = pack2(h[2 * e], h[2 * e + 1]);
                    if (!PACK)
                        lo[t][g][e] = pack2(l[2 * e], l[2 * e + 1]);
                }
            }
    }
    const int blocks = (a.N + 63) / 64;
    for (int b = chunk * kWaves + wave; b < blocks; b += a.chunks * kWaves) {
        const int n0 = 64 * b;
        v4i wv[4][G];
        if (live) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = min(n0 + 16 * (i >> 2) + 4 * j + (i & 3), a.N - 1);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const int c = PACK ? q % ranks : 4 * g + q;
                    wv[j][g] = v4i{0, 0, 0, 0};
                    if (c < ranks && (!PACK || q < 2 * ranks))
                        wv[j][g] = load8(w + (int64_t)n * a.R + 8 * c);
                }
            }
        }
        const int at = n0 + 16 * q, left = a.N - at;
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const bool mine = 16 * t + i < tile.z && left > 0;
            int o[8] = {};
            if (a.base && mine) {
                const uint16_t *p = a.base + token[t] * a.ldb + at;
                const v4i o0 = load8(p, left), o1 = load8(p + 8, left - 8);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    o[e] = o0[e];
                    o[4 + e] = o1[e];
                }
            }
            v4f acc[4] = {};
            if (live)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        acc[j] = mma(wv[j][g], hi[t][g], acc[j]);
                        if (!PACK)
                            acc[j] = mma(wv[j][g], lo[t][PACK ? 0 : g], acc[j]);
                    }
            if (!mine)
                continue;
            if (live || !a.base)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int c = 0; c < 4; c += 2) {
                        const uint32_t d = (uint32_t)o[2 * j + c / 2];
                        o[2 * j + c / 2] = pack2(__uint_as_float(d << 16) + acc[j][c],
                                                 __uint_as_float(d & 0xFFFF0000u) + acc[j][c + 1]);
                    }
            uint16_t *p = a.out + token[t] * a.ldo + at;
            if (left >= 16) {
                __builtin_memcpy(p, o, 32);
            } else {
                uint16_t v[16];
                __builtin_memcpy(v, o, 32);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (e < left)
                        p[e] = v[e];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Gradients
// ---------------------------------------------------------------------------
// out[l][q][p] = in[l][p][q] of the adapters that have tokens; columns P .. ldo - 1 are 0.
struct TransposeArgs {
    const uint16_t *in;
    uint16_t *out;
    const int32_t *offsets;
    int64_t ldo;
    int P, Q;
};

__global__ void __launch_bounds__(kThreads) k_transpose(TransposeArgs a)
{
    __shared__ uint16_t t[64][66];
    const int l = blockIdx.z, q0 = blockIdx.x * 64, p0 = blockIdx.y * 64;
    if (a.offsets[l] == a.offsets[l + 1])
        return;
    const uint16_t *in = a.in + (int64_t)l * a.P * a.Q;
    uint16_t *out = a.out + (int64_t)l * a.Q * a.ldo;
    const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
    for (int p = y; p < 64; p += 4) t[p][x] = p0 + p < a.P && q0 + x < a.Q ? in[(int64_t)(p0 + p) * a.Q + q0 + x] : 0;
    __syncthreads();
    for (int q = y; q < 64; q += 4)
        if (q0 + q < a.Q && p0 + x < a.ldo)
            out[(int64_t)(q0 + q) * a.ldo + p0 + x] = t[x][q];
}

// s v (or s u) as three bf16 pieces, places along the rows: pieces[3][16 RB][places].
struct FactorArgs {
    const float *part, *scale;
    const int32_t *offsets;
    uint16_t *pieces;
    int64_t places;            // of a row, at least tokens
    int tokens, adapters, Rp, splits;
};

__global__ void __launch_bounds__(kThreads) k_factors(FactorArgs a)
{
    __shared__ float t[16][65];
    const int row0 = blockIdx.x * 64, r0 = blockIdx.y * 16, with = a.offsets[a.adapters];
    for (int j = 0; j < 4; ++j) {
        const int r = threadIdx.x & 15, row = row0 + 16 * j + (int)(threadIdx.x >> 4);
        float v = 0.0f;
        if (row < with) {
            for (int k = 0; k < a.splits; ++k) v += a.part[((int64_t)k * a.tokens + row) * a.Rp + r0 + r];
            if (a.scale) {
                int lo = 0, hi = a.adapters;   // the adapter whose places hold the row
                while (hi - lo > 1) {
                    const int m = (lo + hi) / 2;
                    if (a.offsets[m] <= row)
                        lo = m;
                    else
                        hi = m;
                }
                v *= a.scale[lo];
            }
        }
        t[r][row - row0] = v;
    }
    __syncthreads();
    const int r = threadIdx.x >> 4, c = 4 * (threadIdx.x & 15);
    uint16_t o[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float v = t[r][c + i], h = cut(v), m = rest(v, h), mh = cut(m);
        o[0][i] = bf16_bits(h);
        o[1][i] = bf16_bits(mh);
        o[2][i] = bf16_bits(rest(m, mh));
    }
    // (rows of whole 64s: nothing lies behind them)
#pragma unroll
    for (int h = 0; h < 3; ++h)
        __builtin_memcpy(a.pieces + ((int64_t)h * a.Rp + r0 + r) * a.places + row0 + c, o[h], 8);
}

// out[l][r][c] (or [l][c][r]) = sum over the adapter's places of f[r][place] z[token][c].  A wave takes 128
// columns and 16 RB ranks, 32 places at a time: a lane loads 8 columns of 8 tokens and pairs them up for the
// matrix cores, whose m-th product has the columns 8 i + m.  Waves and splits share the places.
struct OuterArgs {
    const uint16_t *z, *pieces;
    const int32_t *order, *offsets;
    float *out;                // [splits] of the result
    int64_t ldz, places, size; // size: elements of the result
    int C, R, Rp, blocks, groups, splits;
    int rank_last;             // the result is [l][c][r]
};

template <int RB>
__global__ void __launch_bounds__(kThreads) k_outer(OuterArgs a)
{
    __shared__ v4f sums[RB * 8][64];
    int b = blockIdx.x;
    const int split = b % a.splits;
    b /= a.splits;
    const int group = b % a.groups;
    b /= a.groups;
    const int c0 = b % a.blocks * 128, l = b / a.blocks;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    const int beg = a.offsets[l], end = a.offsets[l + 1], r0 = group * 16 * RB;
    const int left = a.C - (c0 + 8 * i);
    const uint16_t *z = a.z + c0 + 8 * i;
    v4f acc[RB][8] = {};
    for (int t = beg + 32 * (split * kWaves + wave); t < end; t += 32 * kWaves * a.splits) {
        const int first = t + 8 * q, n = end - first;          // this lane's places
        v4i row[8], f[3][RB];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            row[j] = v4i{0, 0, 0, 0};
            if (j < n)
                row[j] = load8(z + a.order[first + j] * a.ldz, left);
        }
#pragma unroll
        for (int h = 0; h < 3; ++h)
#pragma unroll
            for (int r = 0; r < RB; ++r)
                f[h][r] = load8(a.pieces + ((int64_t)h * a.Rp + r0 + 16 * r + i) * a.places + first, n);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            v4i col;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                col[j] = (int)__builtin_amdgcn_perm((uint32_t)row[2 * j + 1][m / 2], (uint32_t)row[2 * j][m / 2],
                                                    m % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
            for (int h = 0; h < 3; ++h)
#pragma unroll
                for (int r = 0; r < RB; ++r) acc[r][m] = mma(f[h][r], col, acc[r][m]);
        }
    }
    for (int w = 1; w < kWaves; ++w) {
        if (wave == w)
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int m = 0; m < 8; ++m) sums[r * 8 + m][lane] = acc[r][m];
        __syncthreads();
        if (wave == 0)
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int m = 0; m < 8; ++m) acc[r][m] += sums[r * 8 + m][lane];
        __syncthreads();
    }
    if (wave > 0)
        return;
    float *out = a.out + split * a.size;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        const int rank = r0 + 16 * r + 4 * q;
        if (rank >= a.R)
            continue;
        if (a.rank_last) {
#pragma unroll
            for (int m = 0; m < 8; ++m)
                if (m < left)
                    __builtin_memcpy(out + ((int64_t)l * a.C + c0 + 8 * i + m) * a.R + rank, &acc[r][m], 16);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float *o = out + ((int64_t)l * a.R + rank + c) * a.C + c0 + 8 * i;
                float v[8];
#pragma unroll
                for (int m = 0; m < 8; ++m) v[m] = acc[r][m][c];
                if (left >= 8) {
                    __builtin_memcpy(o, v, 32);
                } else {
#pragma unroll
                    for (int m = 0; m < 8; ++m)
                        if (m < left)
                            o[m] = v[m];
                }
            }
        }
    }
}

// out = the splits' parts, added in order.
__global__ void __launch_bounds__(kThreads) k_add_parts(float *out, const float *part, int64_t size, int splits)
{
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < size; i += step) {
        float v = 0.0f;
        for (int k = 0; k < splits; ++k) v += part[k * size + i];
        out[i] = v;
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
struct Sizes {
    int64_t T, K, N, R, L;
    int rb, tb, max_tiles;     // blocks of 16 ranks (1, 2, 4 or 8) and of 16 tokens of a tile
    int64_t Rp;
};

Sizes sizes(int64_t T, int64_t K, int64_t N, int64_t R, int64_t L)
{
    Sizes z{T, K, N, R, L, 1, 1, 0, 0};
    while (16 * z.rb < R) z.rb *= 2;
    z.Rp = 16 * z.rb;
    // tiles as full as the adapters' mean number of tokens lets them be, at most 8 products of accumulators
    const int64_t mean = T / std::min(L, std::max<int64_t>(T, 1));
    while (z.tb < 4 && z.tb * z.rb < 8 && mean > 16 * z.tb) z.tb *= 2;
    z.max_tiles = (int)std::max<int64_t>(1, T / (16 * z.tb) + std::min(L + 1, T));
    return z;
}

int shrink_splits(const Sizes &z, int64_t K)
{
    const int64_t steps = (K + kStep - 1) / kStep, most = (steps + kWaves - 1) / kWaves;
    return (int)std::max<int64_t>(1, std::min<int64_t>({most, 32, 2048 / z.max_tiles}));
}

int outer_splits(const Sizes &z, int64_t C)
{
    const int64_t wgs = z.L * ((C + 127) / 128) * (z.rb > 4 ? 2 : 1);
    return (int)std::max<int64_t>(1, std::min<int64_t>({512 / wgs, z.T / 512, 16}));
}

// Consecutive pieces of the workspace, 256-byte aligned.
struct Layout {
    uint8_t *base;
    size_t bytes = 0;
    template <typename T> T *take(int64_t n)
    {
        T *p = reinterpret_cast<T *>(base + bytes);
        bytes += ((size_t)n * sizeof(T) + 255) / 256 * 256;
        return p;
    }
};

struct Forward {
    int32_t *order, *offsets;
    int4 *tiles;
    float *part;
    size_t bytes;
};

Forward forward_space(const Sizes &z, void *ws)
{
    Layout l{static_cast<uint8_t *>(ws)};
    Forward f;
    f.order = l.take<int32_t>(z.T);
    f.offsets = l.take<int32_t>(z.L + 1);
    f.tiles = l.take<int4>(z.max_tiles);
    f.part = l.take<float>(shrink_splits(z, z.K) * z.T * z.Rp);
    f.bytes = l.bytes;
    return f;
}

struct Backward {
    Forward f;                 // its part: v
    float *u, *outer;
    uint16_t *at, *bt, *fv, *fu;
    int64_t ldbt, places;
    size_t bytes;
};

Backward backward_space(const Sizes &z, void *ws)
{
    Backward b;
    b.f = forward_space(z, ws);
    Layout l{static_cast<uint8_t *>(ws), b.f.bytes};
    b.u = l.take<float>(shrink_splits(z, z.N) * z.T * z.Rp);
    b.ldbt = (z.N + 7) / 8 * 8;
    b.at = l.take<uint16_t>(z.L * z.K * z.R);
    b.bt = l.take<uint16_t>(z.L * z.R * b.ldbt);
    b.places = (z.T + 63) / 64 * 64;
    b.fv = l.take<uint16_t>(3 * z.Rp * b.places);
    b.fu = l.take<uint16_t>(3 * z.Rp * b.places);
    const int64_t sa = outer_splits(z, z.K), sb = outer_splits(z, z.N);
    b.outer = l.take<float>(std::max(sa > 1 ? sa * z.L * z.R * z.K : 0, sb > 1 ? sb * z.L * z.R * z.N : 0));
    b.bytes = l.bytes;
    return b;
}

bool good_shape(int64_t T, int64_t K, int64_t N, int64_t R, int64_t L)
{
    return T >= 0 && T <= kMaxTokens && K > 0 && K <= kMaxWidth && N >= 0 && N <= kMaxWidth && R > 0 && R <= kMaxRank &&
           R % 8 == 0 && L > 0 && L <= kMaxAdapters && L * std::max<int64_t>(R, 64) * std::max(K, N) < (int64_t)1 << 35;
}

hipError_t launch_plan(const Sizes &z, const Forward &f, const void *ids, int32_t id_bits, hipStream_t s)
{
    const Plan p{ids, f.order, f.offsets, f.tiles, (int)z.T, (int)z.L, 16 * z.tb, z.max_tiles, id_bits};
    hipLaunchKernelGGL(k_plan, dim3(1), dim3(kPlanThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_shrink(const Sizes &z, const Forward &f, const uint16_t *x, int64_t ldx, const uint16_t *w, int64_t ldw,
                         int64_t K, float *part, hipStream_t s)
{
    const ShrinkArgs a{x, w, f.order, f.tiles, part, ldx, ldw, (int)z.T, (int)K, (int)z.R, shrink_splits(z, K)};
    const dim3 grid((unsigned)(z.max_tiles * a.splits)), block(kThreads);
    switch (z.rb * 8 + z.tb) {
    case 8 + 1: hipLaunchKernelGGL((k_shrink<1, 1>), grid, block, 0, s, a); break;
    case 8 + 2: hipLaunchKernelGGL((k_shrink<2, 1>), grid, block, 0, s, a); break;
    case 8 + 4: hipLaunchKernelGGL((k_shrink<4, 1>), grid, block, 0, s, a); break;
    case 16 + 1: hipLaunchKernelGGL((k_shrink<1, 2>), grid, block, 0, s, a); break;
    case 16 + 2: hipLaunchKernelGGL((k_shrink<2, 2>), grid, block, 0, s, a); break;
    case 16 + 4: hipLaunchKernelGGL((k_shrink<4, 2>), grid, block, 0, s, a); break;
    case 32 + 1: hipLaunchKernelGGL((k_shrink<1, 4>), grid, block, 0, s, a); break;
    case 32 + 2: hipLaunchKernelGGL((k_shrink<2, 4>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((k_shrink<1, 8>), grid, block, 0, s, a); break;
    }
    return hipGetLastError();
}

template <int TB>
void expand_ranks(const ExpandArgs &a, dim3 grid, hipStream_t s)
{
    const dim3 block(kThreads);
    if (a.R <= 16)
        hipLaunchKernelGGL((k_expand<TB, 1, true>), grid, block, 0, s, a);
    else if (a.R <= 32)
        hipLaunchKernelGGL((k_expand<TB, 1, false>), grid, block, 0, s, a);
    else if (TB < 4 && a.R <= 64)
        hipLaunchKernelGGL((k_expand<TB < 4 ? TB : 1, 2, false>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((k_expand<1, 4, false>), grid, block, 0, s, a);
}

hipError_t launch_expand(const Sizes &z, const Forward &f, const float *part, int splits, const float *scale,
                         const uint16_t *w, int64_t N, const uint16_t *base, int64_t ldb, uint16_t *out, int64_t ldo,
                         hipStream_t s)
{
    const int64_t blocks = (N + 63) / 64, full = (blocks + kWaves - 1) / kWaves;
    const int chunks = (int)std::max<int64_t>(1, std::min<int64_t>(full, 4096 / z.max_tiles));
    const ExpandArgs a{part, scale, f.order, f.tiles, w, base, out, ldb, ldo, (int)z.T, (int)N, (int)z.R, (int)z.Rp,
                       splits, chunks};
    const dim3 grid((unsigned)(z.max_tiles * chunks));
    if (z.tb == 4)
        expand_ranks<4>(a, grid, s);
    else if (z.tb == 2)
        expand_ranks<2>(a, grid, s);
    else
        expand_ranks<1>(a, grid, s);
    return hipGetLastError();
}

hipError_t launch_outer(const Sizes &z, const Backward &b, const uint16_t *x, int64_t ldx, int64_t C,
                        const uint16_t *pieces, bool rank_last, float *out, hipStream_t s)
{
    const int splits = outer_splits(z, C), rb = std::min(z.rb, 4);
    OuterArgs a{x, pieces, b.f.order, b.f.offsets, splits > 1 ? b.outer : out, ldx, b.places, z.L * z.R * C, (int)C,
                (int)z.R, (int)z.Rp, (int)((C + 127) / 128), z.rb / rb, splits, rank_last};
    const dim3 grid((unsigned)(z.L * a.blocks * a.groups * splits)), block(kThreads);
    if (rb == 1)
        hipLaunchKernelGGL((k_outer<1>), grid, block, 0, s, a);
    else if (rb == 2)
        hipLaunchKernelGGL((k_outer<2>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((k_outer<4>), grid, block, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || splits == 1)
        return e;
    hipLaunchKernelGGL(k_add_parts, dim3((unsigned)std::min<int64_t>((a.size + kThreads - 1) / kThreads, 4096)), block, 0,
                       s, out, b.outer, a.size, splits);
    return hipGetLastError();
}

hipError_t launch_transpose(const Sizes &z, const Forward &f, const uint16_t *in, int64_t P, int64_t Q, uint16_t *out,
                            int64_t ldo, hipStream_t s)
{
    const TransposeArgs a{in, out, f.offsets, ldo, (int)P, (int)Q};
    hipLaunchKernelGGL(k_transpose, dim3((unsigned)((Q + 63) / 64), (unsigned)((ldo + 63) / 64), (unsigned)z.L),
                       dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_factors(const Sizes &z, const Backward &b, const float *part, int splits, const float *scale,
                          uint16_t *pieces, hipStream_t s)
{
    const FactorArgs a{part, scale, b.f.offsets, pieces, b.places, (int)z.T, (int)z.L, (int)z.Rp, splits};
    hipLaunchKernelGGL(k_factors, dim3((unsigned)(b.places / 64), (unsigned)z.rb), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

size_t qlin_lora_workspace_size(int64_t tokens, int64_t K, int64_t N, int64_t rank, int64_t adapters)
{
    if (!good_shape(tokens, K, N, rank, adapters) || tokens == 0)
        return 0;
    return forward_space(sizes(tokens, K, N, rank, adapters), nullptr).bytes;
}

qlin_status qlin_lora_mm(int32_t id_bits, int64_t tokens, int64_t K, int64_t N, int64_t rank, int64_t adapters,
                         const uint16_t *X, int64_t ldx, const uint16_t *A, const uint16_t *B, const void *ids,
                         const float *scale, const uint16_t *base, int64_t ldb, uint16_t *Y, int64_t ldy,
                         void *workspace, size_t workspace_bytes, void *stream)
{
    if (id_bits != 32 && id_bits != 64)
        return QLIN_ERR_BAD_ARGUMENT;
    if (!good_shape(tokens, K, N, rank, adapters))
        return QLIN_ERR_BAD_SHAPE;
    if (tokens == 0 || N == 0)
        return QLIN_OK;
    if (!X || !A || !B || !ids || !Y)
        return QLIN_ERR_NULL_POINTER;
    if (ldx < K || ldx > kMaxStride || ldy < N || ldy > kMaxStride || (base && (ldb < N || ldb > kMaxStride)))
        return QLIN_ERR_BAD_STRIDE;
    if (!aligned(X, 2) || !aligned(A, 2) || !aligned(B, 2) || !aligned(base, 2) || !aligned(Y, 2) ||
        !aligned(ids, id_bits / 8) || !aligned(scale, 4) || !aligned(workspace, 16))
        return QLIN_ERR_MISALIGNED;
    const Sizes z = sizes(tokens, K, N, rank, adapters);
    const Forward f = forward_space(z, workspace);
    if (!workspace || workspace_bytes < f.bytes)
        return QLIN_ERR_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (launch_plan(z, f, ids, id_bits, s) != hipSuccess ||
        launch_shrink(z, f, X, ldx, A, K, K, f.part, s) != hipSuccess ||
        launch_expand(z, f, f.part, shrink_splits(z, K), scale, B, N, base, ldb, Y, ldy, s) != hipSuccess)
        return QLIN_ERR_HIP;
    return QLIN_OK;
}

size_t qlin_lora_backward_workspace_size(int64_t tokens, int64_t K, int64_t N, int64_t rank, int64_t adapters)
{
    if (!good_shape(tokens, K, N, rank, adapters) || N == 0)
        return 0;
    return backward_space(sizes(tokens, K, N, rank, adapters), nullptr).bytes;
}

qlin_status qlin_lora_mm_backward(int32_t id_bits, int64_t tokens, int64_t K, int64_t N, int64_t rank, int64_t adapters,
                                  const uint16_t *dY, int64_t lddy, const uint16_t *X, int64_t ldx, const uint16_t *A,
                                  const uint16_t *B, const void *ids, const float *scale, const uint16_t *base,
                                  int64_t ldb, uint16_t *dX, int64_t lddx, float *dA, float *dB, void *workspace,
                                  size_t workspace_bytes, void *stream)
{
    if (id_bits != 32 && id_bits != 64)
        return QLIN_ERR_BAD_ARGUMENT;
    if (!good_shape(tokens, K, N, rank, adapters) || N == 0)
        return QLIN_ERR_BAD_SHAPE;
    if (!A || !B || !dA || !dB || (tokens > 0 && (!dY || !X || !ids || !dX)))
        return QLIN_ERR_NULL_POINTER;
    if (tokens > 0 && (ldx < K || ldx > kMaxStride || lddy < N || lddy > kMaxStride || lddx < K || lddx > kMaxStride ||
                       (base && (ldb < K || ldb > kMaxStride))))
        return QLIN_ERR_BAD_STRIDE;
    if (!aligned(dY, 2) || !aligned(X, 2) || !aligned(A, 2) || !aligned(B, 2) || !aligned(base, 2) || !aligned(dX, 2) ||
        !aligned(dA, 4) || !aligned(dB, 4) || !aligned(ids, id_bits / 8) || !aligned(scale, 4) || !aligned(workspace, 16))
        return QLIN_ERR_MISALIGNED;
    const Sizes z = sizes(tokens, K, N, rank, adapters);
    const Backward b = backward_space(z, workspace);
    if (!workspace || workspace_bytes < b.bytes)
        return QLIN_ERR_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (launch_plan(z, b.f, ids, id_bits, s) != hipSuccess)
        return QLIN_ERR_HIP;
    if (tokens > 0) {
        const int sv = shrink_splits(z, K), su = shrink_splits(z, N);
        if (launch_transpose(z, b.f, A, rank, K, b.at, rank, s) != hipSuccess ||
            launch_transpose(z, b.f, B, N, rank, b.bt, b.ldbt, s) != hipSuccess ||
            launch_shrink(z, b.f, X, ldx, A, K, K, b.f.part, s) != hipSuccess ||
            launch_shrink(z, b.f, dY, lddy, b.bt, b.ldbt, N, b.u, s) != hipSuccess ||
            launch_factors(z, b, b.f.part, sv, scale, b.fv, s) != hipSuccess ||
            launch_factors(z, b, b.u, su, scale, b.fu, s) != hipSuccess ||
            launch_expand(z, b.f, b.u, su, scale, b.at, K, base, ldb, dX, lddx, s) != hipSuccess)
            return QLIN_ERR_HIP;
    }
    if (launch_outer(z, b, X, ldx, K, b.fu, false, dA, s) != hipSuccess ||
        launch_outer(z, b, dY, lddy, N, b.fv, true, dB, s) != hipSuccess)
        return QLIN_ERR_HIP;
    return QLIN_OK;
}

}  // extern "C"
