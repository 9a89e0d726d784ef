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
// v and u stay fp32 between them.  A matrix core takes them as three bf16 pieces, which
// are all of their 24 bits: the upper 16 bits (cut, so that nothing overflows), of the
// rest the upper 16 bits, and what is left.
// Two pieces, 16 bits, would do for y and dx but where base and product cancel, and cost
// less: 8192 tokens of 8 adapters of 64 ranks, K = N = 5120, 113 us for 116.
#include <algorithm>

#include "qlin_device.h"
#include "qlin_overlap.h"
#include "qlin_sort.h"
#include "qlinear.h"

namespace qlin {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kMaxAdapters = 2047;
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

__device__ inline void store8(uint16_t *p, v4i v, int n)
{
    if (n >= 8) {
        __builtin_memcpy(p, &v, 16);
        return;
    }
    uint16_t t[8];
    __builtin_memcpy(t, &v, 16);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n)
            p[i] = t[i];
}

constexpr int kPieces = 3;

// The pieces of v as the upper halves of floats (the last one has eight bits left, too).  Where nothing is left of v, and
// for an infinity, 2^-40 of v stands for the rest: with zero, an infinity among the weights would come out as NaN (as it
// does with a v below 2^-86, whose 2^-40 are no bf16 number any more).  All pieces have v's sign.
__device__ inline void pieces_of(float (&p)[kPieces], float v)
{
    const float least = v * 0x1p-40f;
    float r = v;
#pragma unroll
    for (int h = 0; h < kPieces - 1; ++h) {
        p[h] = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u);
        r -= p[h];
        r = __builtin_amdgcn_classf(r, 0x63) ? least : r;    // NaN or zero
    }
    p[kPieces - 1] = r;
}

__device__ inline uint16_t upper_half(float v) { return (uint16_t)(__float_as_uint(v) >> 16); }

__device__ inline int upper_halves(float lo, float hi)
{
    return (int)__builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

__device__ inline int pack2(float lo, float hi)
{
    return (int)((uint32_t)bf16_bits(lo) | (uint32_t)bf16_bits(hi) << 16);
}

// ---------------------------------------------------------------------------
// Plan: tokens by adapter, and the tiles of each.
// ---------------------------------------------------------------------------
constexpr int kBins = kMaxAdapters + 1;        // the last one in use: tokens without an adapter

struct Plan {
    const void *ids;
    int32_t *order;            // [tokens]: the tokens by (adapter, token); those without one come last
    int32_t *offsets;          // [adapters + 1]: the first place of each adapter (NULL: not wanted)
    int4 *tiles;               // [max_tiles]: adapter (-1: none), first place, tokens (0: no tile), and the
                               // tokens of the expand tile that begins here (0: none does)
    int4 *wides;               // [max_wides]: the tiles where an expand tile begins (NULL: not wanted); without it
                               // the others' workgroups of the expand kernel, which have no work, cost it up to 3 us
    int tokens, adapters, tile, wide, max_tiles, max_wides, id_bits;
};

__device__ inline int bin_of(const Plan &p, int t)
{
    const int64_t id = p.id_bits == 64 ? static_cast<const int64_t *>(p.ids)[t] : static_cast<const int32_t *>(p.ids)[t];
    return id >= 0 && id < p.adapters ? (int)id : p.adapters;
}

// Tile j of an adapter with n tokens from place `first`.
__device__ inline int4 tile_of(const Plan &p, int bin, int first, int n, int j)
{
    const int at = j * p.tile;
    return make_int4(bin < p.adapters ? bin : -1, first + at, min(p.tile, n - at),
                     at % p.wide == 0 ? min(p.wide, n - at) : 0);
}

// Adds the wave's bins (-1: none) to its counts; where all are one request's, with one addition.
__device__ inline void count_bins(int32_t *hist, int bin, int lane)
{
    const uint64_t any = __ballot(bin >= 0);
    if (!any)
        return;
    const int lead = __ffsll((unsigned long long)any) - 1, b = __builtin_amdgcn_readlane(bin, lead);
    if (__ballot(bin == b) == any) {
        if (lane == lead)
            atomicAdd(&hist[b], __popcll(any));
    } else if (bin >= 0) {
        atomicAdd(&hist[bin], 1);
    }
}

// More than 8192 tokens: a counting sort over several workgroups, the last of which writes the tiles (65536 tokens:
// 14 us).
struct ManyArgs {
    Plan plan;
    SortRange range;
    int digits;                // a power of two above the number of adapters
};

__global__ void __launch_bounds__(kSortThreads) k_plan_count(ManyArgs a)
{
    extern __shared__ int32_t hist[];
    count(a.range, 0, a.digits, hist, [&](int i) { return bin_of(a.plan, i); });
}

__global__ void __launch_bounds__(kSortThreads) k_plan_place(ManyArgs a)
{
    extern __shared__ int32_t hist[];
    const Plan &p = a.plan;
    place(a.range, 0, a.digits, hist, [&](int i) { return make_int2(bin_of(p, i), i); },
          [&](int at, int2 t) { p.order[at] = t.y; });
    if (blockIdx.x != gridDim.x - 1)
        return;
    const int32_t *total = hist + kSortWaves * a.digits;
    const int lane = threadIdx.x & 63;
    int at0 = 0, tile0 = 0, wide0 = 0;
    for (int b0 = 0; b0 <= p.adapters; b0 += 64) {          // (by each wave, which takes its share of the tiles)
        const int b = b0 + lane, n = b <= p.adapters ? total[b] : 0, tiles = (n + p.tile - 1) / p.tile;
        const int at = at0 + wave_scan(n) - n, tile = tile0 + wave_scan(tiles) - tiles;
        const int wides = (n + p.wide - 1) / p.wide, wide = wide0 + wave_scan(wides) - wides;
        if (b <= p.adapters) {
            if (p.offsets && threadIdx.x < 64)
                p.offsets[b] = at;             // (that of the last bin: tokens with an adapter)
            for (int j = threadIdx.x >> 6; j < tiles; j += kSortWaves) {
                const int4 t = tile_of(p, b, at, n, j);
                p.tiles[tile + j] = t;
                if (p.wides && t.w)
                    p.wides[wide + j * p.tile / p.wide] = t;
            }
        }
        at0 = __builtin_amdgcn_readlane(at + n, 63);
        tile0 = __builtin_amdgcn_readlane(tile + tiles, 63);
        wide0 = __builtin_amdgcn_readlane(wide + wides, 63);
    }
    for (int t = tile0 + (int)threadIdx.x; t < p.max_tiles; t += kSortThreads) p.tiles[t] = make_int4(-1, 0, 0, 0);
    if (p.wides)
        for (int t = wide0 + (int)threadIdx.x; t < p.max_wides; t += kSortThreads) p.wides[t] = make_int4(-1, 0, 0, 0);
}

// Up to 64 tokens: every wave of the shrink kernel finds its tile by itself, without LDS or a barrier.  `token`
// becomes the token at the lane's place.
constexpr int kWaveTokens = 64;

__device__ inline int4 wave_plan(const Plan &p, int want, int &token)
{
    const int lane = threadIdx.x & 63;
    const int bin = lane < p.tokens ? bin_of(p, lane) : kBins;
    int place = 0;
    for (int j = 0; j < p.tokens; ++j) {
        const int o = __builtin_amdgcn_readlane(bin, j);
        place += o < bin || (o == bin && j < lane) ? 1 : 0;
    }
    token = __builtin_amdgcn_ds_permute(4 * place, lane);
    const int sorted = __builtin_amdgcn_ds_permute(4 * place, bin);
    const int ahead = __shfl_up(sorted, 1);                 // (by all lanes)
    const bool there = lane < p.tokens, starts = there && (lane == 0 || ahead != sorted);
    const uint64_t firsts = __ballot(starts), low = ((uint64_t)2 << lane) - 1;
    const int first = 63 - __clzll((long long)(firsts & low));
    const uint64_t heads = __ballot(there && (lane - first) % p.tile == 0);
    const uint64_t mine = __ballot(((heads >> lane) & 1) && __popcll(heads & (low >> 1)) == want);
    if (want == 0 && p.offsets)
        for (int b0 = 0; b0 <= p.adapters; b0 += blockDim.x) {         // (by all lanes: other lanes' bins are read)
            const int b = b0 + threadIdx.x;
            int n = 0;
            for (int j = 0; j < p.tokens; ++j) n += __builtin_amdgcn_readlane(bin, j) < b ? 1 : 0;
            if (b <= p.adapters)
                p.offsets[b] = n;
        }
    if (!mine)
        return make_int4(-1, 0, 0, 0);
    const int at = __ffsll((unsigned long long)mine) - 1, begin = __builtin_amdgcn_readlane(first, at);
    const uint64_t later = firsts & ~(((uint64_t)2 << begin) - 1);
    const int end = later ? __ffsll((unsigned long long)later) - 1 : p.tokens;
    return tile_of(p, __builtin_amdgcn_readlane(sorted, at), begin, end - begin, (at - begin) / p.tile);
}

// Up to 8192: every workgroup of the shrink kernel finds its tile (4 us for 4001 tokens; the two launches above take 14).
// A wave owns a contiguous part of the tokens, keeps their bins and counts them for itself; then each wave walks the bins,
// 64 at a time.
constexpr int kHold = 16;
constexpr int kSelfTokens = 64 * 8 * kHold;

// The tile `want`; its tokens in `token` (LDS); `hist` [waves][adapters + 1] (LDS).  Called by all threads.  With `publish`
// it goes to the plan's lists.
__device__ inline int4 self_plan(const Plan &p, int want, int32_t *hist, int32_t *token, bool publish)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6, bins = p.adapters + 1;
    const int turns = (p.tokens + (int)blockDim.x - 1) / (int)blockDim.x, beg = wave * turns * 64 + lane;
    int held[kHold];
#pragma unroll
    for (int h = 0; h < kHold; ++h) held[h] = h < turns && beg + 64 * h < p.tokens ? bin_of(p, beg + 64 * h) : -1;
    int32_t *mine = hist + wave * bins;
    for (int b = lane; b < bins; b += 64) mine[b] = 0;
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
        if (h >= turns)
            break;
        count_bins(mine, held[h], lane);
    }
    __syncthreads();
    int4 found = make_int4(-1, 0, 0, 0);
    int bin = -1, skip = 0, wide0 = 0, at_wide = 0;
    const bool offsets = want == 0 && wave == 0 && p.offsets, all = offsets || (wave == 0 && publish && p.wides);
    for (int b0 = 0, at0 = 0, tile0 = 0; b0 < bins && (all || bin < 0); b0 += 64) {
        int n = 0;
        if (b0 + lane < bins)
            for (int w = 0; w < waves; ++w) n += hist[w * bins + b0 + lane];
        const int tiles = (n + p.tile - 1) / p.tile, at = at0 + wave_scan(n) - n, tile = tile0 + wave_scan(tiles) - tiles;
        const int wides = (n + p.wide - 1) / p.wide, wide = wide0 + wave_scan(wides) - wides;
        if (offsets && b0 + lane < bins)
            p.offsets[b0 + lane] = at;
        const uint64_t here = __ballot(want >= tile && want < tile + tiles);
        if (here) {
            const int l = __ffsll((unsigned long long)here) - 1, j = want - __builtin_amdgcn_readlane(tile, l);
            bin = b0 + l;
            skip = j * p.tile;
            found = tile_of(p, bin, __builtin_amdgcn_readlane(at, l), __builtin_amdgcn_readlane(n, l), j);
            at_wide = __builtin_amdgcn_readlane(wide, l) + skip / p.wide;
        }
        at0 = __builtin_amdgcn_readlane(at + n, 63);
        tile0 = __builtin_amdgcn_readlane(tile + tiles, 63);
        wide0 = __builtin_amdgcn_readlane(wide + wides, 63);
    }
    if (publish && threadIdx.x == 0) {
        p.tiles[want] = found;
        if (p.wides && found.w)
            p.wides[at_wide] = found;
        if (p.wides && want >= wide0 && want < p.max_wides)
            p.wides[want] = make_int4(-1, 0, 0, 0);
    }
    if (bin < 0)
        return found;                          // (in all waves)
    int rank = -skip;
    for (int w = 0; w < wave; ++w) rank += hist[w * bins + bin];
    const int here = hist[wave * bins + bin];
    if (rank < found.z && rank + here > 0)
#pragma unroll
        for (int h = 0; h < kHold; ++h) {
            if (h >= turns)
                break;
            const uint64_t same = __ballot(held[h] == bin);
            const int r = rank + __popcll(same & (((uint64_t)1 << lane) - 1));
            if (held[h] == bin && r >= 0 && r < found.z)
                token[r] = beg + 64 * h;
            rank += __popcll(same);
        }
    __syncthreads();
    return found;
}

// ---------------------------------------------------------------------------
// Shrink: s v[place,r] with v = sum_k x[token,k] w[adapter,r,k], or, where the weights lie as [k][r], the
// same from them (u).  Sixteen tokens by sixteen ranks a matrix product; a workgroup has a tile and all of
// K, which its waves share in steps of 64 and add up in LDS.  Weights as [k][r] go through LDS, whose
// transposing loads give a lane eight k of its rank.
//
// The lines of 128 bytes that a CU asks of the L2 bound it, about 160 a microsecond, the weights' of every tile
// among them: u and v of 8192 tokens of 5120 and 10240, 16 ranks, 3.0 million, 79 us (140 a CU and microsecond); 4001
// tokens of 6 adapters of 32 ranks, K = 5120, 1.0 million lines, 21 us (122: a workgroup a CU, and nothing covers its
// plan, 4 us, and its sums).  Tiles of 64 tokens with K in parts, a launch that adds them, need a tenth fewer lines
// and took 67 us for the former, but 25 us more for the plan and the parts.
// ---------------------------------------------------------------------------
constexpr int kStep = 64;

struct ShrinkJob {
    const uint16_t *x, *w;
    float *sums;               // [splits][tokens][Rp]: sums of parts of K, without s, for expand (or NULL)
    uint16_t *pieces;          // [place / 8][3][Rp][8]: the pieces, for outer (or NULL)
    int64_t ldx;
    int K;
};

struct ShrinkArgs {
    ShrinkJob job[2];          // v; u
    Plan plan;
    const float *scale;
    int splits;                // parts of K (backward: 1)
    int R, Rp, groups, self;   // groups of 16 RB ranks; self: waves (1) or workgroups (2) make the plan
};

// Waves of a workgroup (16 took as long, four 39 us for 35: the gradients of 2048 tokens of an adapter of 16 ranks,
// K = N = 2048), and steps whose loads a wave has in flight.
constexpr int kShrinkWaves = 8;
template <int TB, int RB> constexpr int steps_at_once() { return TB * RB == 1 ? 5 : TB + RB <= 3 ? 3 : TB + RB <= 5 ? 2 : 1; }

// A step's rows: eight lanes load 128 bytes of one, so that a load instruction touches eight lines (with a row
// for each lane of sixteen, as the matrix cores want them, it touches 64: 32 tokens of 28 adapters on K = 5120
// took 12.4 us, so 10.4).  The wave's LDS brings them to the matrix cores' order; piece j of a row lies at j ^ row, which
// keeps both directions free of bank conflicts.
template <int B>
__device__ inline void load_rows(v4i (&v)[B][2], const uint16_t *const (&p)[B][2], int k, int K)
{
    if (k + kStep <= K) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
            v[b][0] = load8(p[b][0] + k);
            v[b][1] = load8(p[b][1] + k);
        }
    } else {
        const int left = K - (k + 8 * (threadIdx.x & 7));
#pragma unroll
        for (int b = 0; b < B; ++b) {
            v[b][0] = load8(p[b][0] + k, left);
            v[b][1] = load8(p[b][1] + k, left);
        }
    }
}

template <int B>
__device__ inline void store_rows(v4i *lds, const v4i (&v)[B][2])
{
    const int lane = threadIdx.x & 63, row = lane >> 3, at = 8 * row + ((lane & 7) ^ row);
#pragma unroll
    for (int b = 0; b < B; ++b) {
        lds[128 * b + at] = v[b][0];
        lds[128 * b + 64 + at] = v[b][1];
    }
}

// Row l % 16 of block b, the half's eight k of the lane's quarter.
__device__ inline v4i row_part(const v4i *lds, int b, int half)
{
    const int lane = threadIdx.x & 63, i = lane & 15;
    return lds[128 * b + 8 * i + ((4 * half + (lane >> 4)) ^ (i & 7))];
}

// Between a wave's stores into LDS and its lanes' loads of what others stored, and back: the LDS takes a wave's accesses
// in order, so that this only keeps the compiler from changing it.
__device__ inline void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Adds the steps first, first + kShrinkWaves, .. before `end` of 16 TB tokens and the ranks from r0 of weights [R][K].
template <int TB, int RB>
__device__ inline void add_steps(v4f (&acc)[TB][RB], const uint16_t *const (&px)[TB][2], const uint16_t *rows, int R, int r0,
                                 int K, int first, int end, v4i *mine)
{
    constexpr int U = steps_at_once<TB, RB>(), waves = kShrinkWaves;
    const int lane = threadIdx.x & 63;
    v4i *const weights = mine + TB * 128;
    const uint16_t *pw[RB][2];                 // (ranks behind R take the last one's row: their sums are not read)
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            pw[r][h] = rows + (int64_t)min(r0 + 16 * r + 8 * h + (lane >> 3), R - 1) * K + 8 * (lane & 7);
    for (int s = first; s < end; s += waves * U) {
        v4i x[U][TB][2], w[U][RB][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u > 0 && s + waves * u >= end)
                break;
            load_rows(x[u], px, (s + waves * u) * kStep, K);
            load_rows(w[u], pw, (s + waves * u) * kStep, K);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u > 0 && s + waves * u >= end)
                break;
            wave_sync();                       // (the step before has been read)
            store_rows(mine, x[u]);
            store_rows(weights, w[u]);
            wave_sync();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4i f[RB];
#pragma unroll
                for (int r = 0; r < RB; ++r) f[r] = row_part(weights, r, h);
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    const v4i y = row_part(mine, t, h);
#pragma unroll
                    for (int r = 0; r < RB; ++r) acc[t][r] = mma(y, f[r], acc[t][r]);
                }
            }
        }
    }
}

// Where the pieces of adapter l's places begin, or of a tile of it (tiles have whole sixteens before them): at
// eights, so that no two adapters share one, whatever their numbers of tokens.
__host__ __device__ inline int64_t piece_place(int64_t place, int l) { return (place + 7) / 8 * 8 + 8 * (int64_t)l; }

// A wave's share of LDS: a step's rows and weights, then its sums (16-byte pieces).
constexpr int shrink_share(int tb, int rb) { return tb * rb > 2 * (tb + rb) ? tb * rb * 64 : 2 * (tb + rb) * 64; }

template <int TB, int RB, bool BACK>
__global__ void __launch_bounds__(64 * kShrinkWaves) k_shrink(ShrinkArgs a)
{
    constexpr int kShare = shrink_share(TB, RB);
    extern __shared__ v4i shared[];            // [waves][kShare], before that the plan's bins
    __shared__ int32_t tokens[64];
    const int units = a.plan.max_tiles * a.groups;
    // (the longer job's workgroups come first)
    const int later = BACK && (int)blockIdx.x >= units, second = BACK && later != (a.job[1].K > a.job[0].K);
    const ShrinkJob &job = a.job[second];
    const int split = BACK ? 0 : (int)blockIdx.x % a.splits;
    const int unit = BACK ? (int)blockIdx.x - (later ? units : 0) : (int)blockIdx.x / a.splits;
    const int index = unit / a.groups, group = unit % a.groups;
    const bool publish = group == 0 && !second && split == 0;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, q = lane >> 4;
    constexpr int waves = kShrinkWaves;
    int4 tile;
    int token[TB];
    if (a.self == 1) {
        int sorted;
        tile = wave_plan(a.plan, index, sorted);
#pragma unroll
        for (int t = 0; t < TB; ++t) token[t] = __shfl(sorted, tile.y + min(16 * t + i, tile.z - 1));
        const int there = __shfl(sorted, (tile.y + lane) & 63);          // (by all lanes)
        if (publish && wave == 0 && lane < tile.z)
            a.plan.order[tile.y + lane] = there;
        if (publish && tid == 0)
            a.plan.tiles[index] = tile;
    } else {
        if (a.self) {
            tile = self_plan(a.plan, index, reinterpret_cast<int32_t *>(shared), tokens, publish);
            if (publish && tid < tile.z)
                a.plan.order[tile.y + tid] = tokens[tid];
#pragma unroll
            for (int t = 0; t < TB; ++t) token[t] = tile.z ? tokens[min(16 * t + i, tile.z - 1)] : 0;
        } else {
            tile = a.plan.tiles[index];
#pragma unroll
            for (int t = 0; t < TB; ++t) token[t] = tile.z ? a.plan.order[tile.y + min(16 * t + i, tile.z - 1)] : 0;
        }
    }
    if (tile.x < 0 || tile.z == 0)
        return;
    const uint16_t *px[TB][2];                 // rows l / 8 and 8 behind of each block
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            px[t][h] = job.x + __shfl(token[t], 8 * h + (lane >> 3)) * job.ldx + 8 * (lane & 7);
    v4f acc[TB][RB] = {};
    const int steps = (job.K + kStep - 1) / kStep, r0 = 16 * RB * group;
    v4i *const mine = shared + wave * kShare, *const weights = mine + TB * 128;
    if (!BACK || !second) {
        const int per = (steps + a.splits - 1) / a.splits, end = min((split + 1) * per, steps);
        add_steps(acc, px, job.w + (int64_t)tile.x * a.R * job.K, a.R, r0, job.K, split * per + wave, end, mine);
    } else {
        // 64 rows of up to 2 RB chunks of 8 ranks a step, one row after another
        const int chunks = min(2 * RB, a.R / 8 - r0 / 8);
        const uint16_t *w = job.w + (int64_t)tile.x * job.K * a.R + r0;
        uint16_t *const wl = reinterpret_cast<uint16_t *>(weights);
        int row[2 * RB], rank[2 * RB];
#pragma unroll
        for (int h = 0; h < 2 * RB; ++h) {
            row[h] = (lane + 64 * h) / chunks;
            rank[h] = 8 * ((lane + 64 * h) % chunks);
        }
        v4i x[TB][2], b[2 * RB];
        const auto load = [&](int s) {
            load_rows(x, px, s * kStep, job.K);
#pragma unroll
            for (int h = 0; h < 2 * RB; ++h) {
                b[h] = v4i{0, 0, 0, 0};
                if (row[h] < kStep && s * kStep + row[h] < job.K)
                    b[h] = load8(w + (int64_t)(s * kStep + row[h]) * a.R + rank[h]);
            }
        };
        if (wave < steps)
            load(wave);
        for (int s = wave; s < steps; s += waves) {
            wave_sync();                       // (the step before has been read)
            store_rows(mine, x);
#pragma unroll
            for (int h = 0; h < 2 * RB; ++h)
                if (row[h] < kStep)
                    *reinterpret_cast<v4i *>(wl + row[h] * (16 * RB) + rank[h]) = b[h];
            wave_sync();
            if (s + waves < steps)
                load(s + waves);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4i f[RB];
#pragma unroll
                for (int r = 0; r < RB; ++r)
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        // sixteen lanes load four rows of sixteen ranks, and get a column each
                        typedef short v4s __attribute__((ext_vector_type(4)));
                        uint16_t *p = wl + (32 * h + 8 * q + 4 * g + (i >> 2)) * (16 * RB) + 16 * r + 4 * (i & 3);
                        const v4s v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)p);
                        const int2 d = __builtin_bit_cast(int2, v);
                        f[r][2 * g] = d.x;
                        f[r][2 * g + 1] = d.y;
                    }
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    const v4i y = row_part(mine, t, h);
#pragma unroll
                    for (int r = 0; r < RB; ++r) acc[t][r] = mma(y, f[r], acc[t][r]);
                }
            }
        }
    }
    __syncthreads();                           // (another wave may still read its weights where sums go)
    v4f *sums = reinterpret_cast<v4f *>(shared);
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int r = 0; r < RB; ++r) sums[(wave * TB * RB + t * RB + r) * 64 + lane] = acc[t][r];
    __syncthreads();
    const float s = a.scale ? a.scale[tile.x] : 1.0f;
    for (int e = tid; e < TB * RB * 64; e += 64 * waves) {
        v4f v = sums[e];
        for (int w = 1; w < waves; ++w) v += sums[w * TB * RB * 64 + e];
        const int block = e >> 6, rank = r0 + 16 * (block % RB) + (e & 15), at = 16 * (block / RB) + 4 * ((e >> 4) & 3);
        const int n = tile.z - at;             // of the four places from there
        if (!BACK || job.sums)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c < n)
                    job.sums[((int64_t)split * a.plan.tokens + tile.y + at + c) * a.Rp + rank] = v[c];
        if (BACK && (at & ~7) < tile.z) {      // (zeros fill the last eight)
            uint16_t o[kPieces][4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float f[kPieces];
                pieces_of(f, c < n ? v[c] * s : 0.0f);
#pragma unroll
                for (int h = 0; h < kPieces; ++h) o[h][c] = upper_half(f[h]);
            }
            const int64_t eight = piece_place(tile.y, tile.x) / 8 + at / 8;
#pragma unroll
            for (int h = 0; h < kPieces; ++h)
                __builtin_memcpy(job.pieces + ((eight * kPieces + h) * a.Rp + rank) * 8 + (at & 4), o[h], 8);
        }
    }
}

// ---------------------------------------------------------------------------
// Expand: out[token,n] = bf16(base[token,n] + sum_r (s v)[place,r] w[adapter,n,r]), or with the weights as
// [adapter][r][n] (dx).  Two kernels: where an adapter has few tokens its weights are what is read, and a wave
// takes them straight into registers; where it has many, base and out are, and the waves of a workgroup, 16
// tokens each, share the weights in LDS.
// ---------------------------------------------------------------------------
constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kWide = 16 * kWaves;             // tokens of a workgroup of the second kernel

struct ExpandArgs {
    const float *sums;         // [splits][tokens][Rp]: the parts of v
    const float *scale;        // s, or NULL
    int tokens, splits;
    const int32_t *order;
    const int4 *tiles;
    const uint16_t *w, *base;
    uint16_t *out;
    int64_t ldb, ldo;
    int N, R, Rp, chunks;
};

// The pieces of s times eight sums.
template <int G>
__device__ inline void cut_factors(v4i (&f)[kPieces][G], int g, const v4f (&sum)[2], float s)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float p0[kPieces], p1[kPieces];
        pieces_of(p0, sum[e / 2][2 * e % 4] * s);
        pieces_of(p1, sum[e / 2][2 * e % 4 + 1] * s);
#pragma unroll
        for (int h = 0; h < kPieces; ++h) f[h][g][e] = upper_halves(p0[h], p1[h]);
    }
}

// The pieces of s v as operands, chunk 4 g + q of 8 ranks, from the parts of v, four of them on their way at a time.  (Cut
// here and not by shrink: two bytes fewer a rank and token to write and to read.)
template <int G>
__device__ inline void load_factors(v4i (&f)[kPieces][G], const ExpandArgs &a, int place, float s)
{
    const int q = (threadIdx.x & 63) >> 4, ranks = a.R / 8;
    const int64_t apart = (int64_t)a.tokens * a.Rp;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int c = 4 * g + q;
#pragma unroll
        for (int h = 0; h < kPieces; ++h) f[h][g] = v4i{0, 0, 0, 0};
        if (c >= ranks)
            continue;
        const float *p = a.sums + (int64_t)place * a.Rp + 8 * c;
        v4f sum[2] = {};
        for (int k = 0; k < a.splits; k += 4) {
            v4f v[4][2] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k + j < a.splits) {
                    v[j][0] = *reinterpret_cast<const v4f *>(p + (k + j) * apart);
                    v[j][1] = *reinterpret_cast<const v4f *>(p + (k + j) * apart + 4);
                }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum[0] += v[j][0];
                sum[1] += v[j][1];
            }
        }
        cut_factors(f, g, sum, s);
    }
}

// 64 n of a wave as four products of 16 n by 16 tokens, dealt to them so that a lane ends with twice eight n
// in a row of its token, and four lanes with 64 bytes of it.
template <int G, bool TR>
struct Few {
    v4i o[2], f[4][G];         // this lane's outputs, n0 + 8 q .. + 7 and 32 behind; operands of the products

    // `w`: the adapter's weights, NULL for none; `row`: the lane's token, -1 for none
    __device__ void load(const ExpandArgs &a, const uint16_t *w, int64_t row, int n0)
    {
        const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
        const int ranks = a.R / 8;             // chunks of 8 ranks
        o[0] = o[1] = v4i{0, 0, 0, 0};
        if (a.base && row >= 0) {
            const uint16_t *p = a.base + row * a.ldb + n0 + 8 * q;
            const int left = a.N - (n0 + 8 * q);
            o[0] = load8(p, left);
            o[1] = load8(p + 32, left - 32);
        }
        if (!w)
            return;
        if (TR) {
            // rows of eight ranks, four n of each: the lane's row 4 a + c of product m is
            // n = 32 (c / 2) + 8 a + 4 (c % 2) + m
            const int n = n0 + 32 * ((i & 3) >> 1) + 8 * (i >> 2) + 4 * (i & 1), there = a.N - n;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int c = 4 * g + q;
                int2 r[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    r[j] = make_int2(0, 0);
                    if (c < ranks) {
                        const uint16_t *p = w + (int64_t)(8 * c + j) * a.N + n;
                        if (there >= 4) {
                            __builtin_memcpy(&r[j], p, 8);
                        } else {
                            uint16_t e[4];
#pragma unroll
                            for (int m = 0; m < 4; ++m) e[m] = m < there ? p[m] : 0;
                            __builtin_memcpy(&r[j], e, 8);
                        }
                    }
                }
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        f[m][g][j] = (int)__builtin_amdgcn_perm(
                            (uint32_t)(m < 2 ? r[2 * j + 1].x : r[2 * j + 1].y),
                            (uint32_t)(m < 2 ? r[2 * j].x : r[2 * j].y), m % 2 ? 0x07060302u : 0x05040100u);
            }
        } else {
            // rows of n: row 4 a + c of product j is n = 32 (j / 2) + 8 a + 4 (j % 2) + c
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = min(n0 + 32 * (j >> 1) + 8 * (i >> 2) + 4 * (j & 1) + (i & 3), a.N - 1);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const int c = 4 * g + q;
                    f[j][g] = v4i{0, 0, 0, 0};
                    if (c < ranks)
                        f[j][g] = load8(w + (int64_t)n * a.R + 8 * c);
                }
            }
        }
    }

    __device__ void add(const v4i (&v)[kPieces][G])
    {
        v4f acc[4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int h = 0; h < kPieces; ++h) acc[j] = mma(f[j][g], v[h][g], acc[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d0 = TR ? acc[(2 * e) % 4][e / 2] : acc[e / 2][(2 * e) % 4];
            const float d1 = TR ? acc[(2 * e + 1) % 4][e / 2] : acc[e / 2][(2 * e + 1) % 4];
            const uint32_t d = (uint32_t)o[e / 4][e % 4];
            o[e / 4][e % 4] = pack2(__uint_as_float(d << 16) + d0, __uint_as_float(d & 0xFFFF0000u) + d1);
        }
    }

    __device__ void store(const ExpandArgs &a, int64_t row, int n0) const
    {
        if (row < 0)
            return;
        const int q = (threadIdx.x & 63) >> 4, left = a.N - (n0 + 8 * q);
        uint16_t *p = a.out + row * a.ldo + n0 + 8 * q;
        store8(p, o[0], left);
        store8(p + 32, o[1], left - 32);
    }
};

// Weights' bytes bound it: 128 tokens of 24 adapters of 64 ranks on N = 51200, 183 MB, 41 us, 4.5 TB/s (with two pieces of
// v, cut by shrink, 37 us; two or four blocks a workgroup, and weights loaded ahead of v, took as long or longer).
template <int G, bool TR>
__global__ void __launch_bounds__(kThreads) k_expand_few(ExpandArgs a)
{
    const int4 tile = a.tiles[blockIdx.x / a.chunks];
    const int chunk = blockIdx.x % a.chunks;
    if (tile.w == 0)
        return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15;
    const bool live = tile.x >= 0;
    const int place = tile.y + min(i, tile.w - 1);
    const int64_t token = i < tile.w ? a.order[place] : -1;
    v4i v[kPieces][G];
    const uint16_t *w = live ? a.w + (int64_t)tile.x * a.N * a.R : nullptr;
    if (live)
        load_factors(v, a, place, a.scale ? a.scale[tile.x] : 1.0f);
    const int blocks = (a.N + 63) / 64;
    for (int b = chunk * kWaves + wave; b < blocks; b += a.chunks * kWaves) {
        Few<G, TR> n;
        n.load(a, w, token, 64 * b);
        if (live)
            n.add(v);
        n.store(a, token, 64 * b);
    }
}

// Few tokens of adapters that are small: both products in one launch, every workgroup with its own sums of all of K for
// the tile whose 512 n it has.  A launch less is worth more than the reads of A by every workgroup while these are one a
// CU at most: a token, 16 ranks, K = N = 2048 5.5 us, in two launches 7.3, and 3 us less of the calling thread's time.
template <int RB>
__global__ void __launch_bounds__(64 * kShrinkWaves) k_both(ShrinkArgs s, ExpandArgs a)
{
    constexpr int kRow = 16 * RB + 4;          // a token's sums (a row's start falls on other banks than the last's)
    extern __shared__ v4i shared[];            // [waves][shrink_share]
    __shared__ __align__(16) float sums[16 * kRow];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    int sorted;
    const int4 tile = wave_plan(s.plan, blockIdx.x / a.chunks, sorted);
    const int there = __shfl(sorted, tile.y + min(i, max(tile.z, 1) - 1));
    if (tile.z == 0)
        return;
    const bool live = tile.x >= 0;
    const int64_t token = i < tile.z ? there : -1;
    const uint16_t *w = live ? a.w + (int64_t)tile.x * a.N * a.R : nullptr;
    const int n0 = 64 * (blockIdx.x % a.chunks * kShrinkWaves + wave);
    Few<1, false> n;
    if (n0 < a.N)
        n.load(a, w, token, n0);               // (on its way meanwhile)
    v4i v[kPieces][1] = {};
    if (live) {
        const ShrinkJob &job = s.job[0];
        const uint16_t *px[1][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) px[0][h] = job.x + __shfl(there, 8 * h + (lane >> 3)) * job.ldx + 8 * (lane & 7);
        v4f acc[1][RB] = {};
        add_steps(acc, px, job.w + (int64_t)tile.x * s.R * job.K, s.R, 0, job.K, wave, (job.K + kStep - 1) / kStep,
                  shared + wave * shrink_share(1, RB));
        __syncthreads();
        v4f *parts = reinterpret_cast<v4f *>(shared);
#pragma unroll
        for (int r = 0; r < RB; ++r) parts[(wave * RB + r) * 64 + lane] = acc[0][r];
        __syncthreads();
        if (threadIdx.x < 64 * RB) {
            v4f t = parts[threadIdx.x];
#pragma unroll
            for (int k = 1; k < kShrinkWaves; ++k) t += parts[k * RB * 64 + threadIdx.x];
#pragma unroll
            for (int c = 0; c < 4; ++c) sums[(4 * q + c) * kRow + 16 * wave + i] = t[c];
        }
        __syncthreads();
        if (q < a.R / 8) {
            const v4f *p = reinterpret_cast<const v4f *>(sums + i * kRow + 8 * q);
            const v4f sum[2] = {p[0], p[1]};
            cut_factors(v, 0, sum, a.scale ? a.scale[tile.x] : 1.0f);
        }
    }
    if (n0 >= a.N)
        return;
    if (live)
        n.add(v);
    n.store(a, token, n0);
}

// 128 n a workgroup at a time, 16 tokens a wave: eight products of 16 tokens by 16 n, the m-th with the n = 8 i + m,
// so that a lane ends with eight n in a row of four tokens, and sixteen lanes with 256 bytes of one (64 bytes of
// each token, as above, took 32 us where this took 25: 4001 tokens on N = 5120, 32 ranks; 23 with the plan's list of
// tiles and three pieces of v, base and out at 3.6 TB/s: a workgroup's loads of order, v, weights and base wait for
// each other).
template <int G, bool TR>
__global__ void __launch_bounds__(kThreads) k_expand_many(ExpandArgs a)
{
    extern __shared__ v4i shared[];            // 128 n's weights
    const int4 tile = a.tiles[blockIdx.x / a.chunks];
    const int chunk = blockIdx.x % a.chunks;
    if (tile.w == 0)
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, q = lane >> 4;
    const int ranks = a.R / 8;                 // chunks of 8 ranks
    const bool live = tile.x >= 0;
    int token[4];                              // tokens 4 q + c of the wave's (-1: none)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int at = 16 * wave + 4 * q + c;
        token[c] = at < tile.w ? a.order[tile.y + at] : -1;
    }
    v4i v[kPieces][G];
    const uint16_t *w = a.w + (int64_t)(live ? tile.x : 0) * a.N * a.R;
    if (live) {
        const int place = tile.y + min(16 * wave + i, tile.w - 1);
        load_factors(v, a, place, a.scale ? a.scale[tile.x] : 1.0f);
    }
    const int blocks = (a.N + 127) / 128;
    for (int b = chunk; b < blocks; b += a.chunks) {
        const int n = 128 * b + 8 * i, left = a.N - n;      // this lane's n .. n + 7
        v4i o[4] = {};
        if (a.base)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (token[c] >= 0)
                    o[c] = load8(a.base + token[c] * a.ldb + n, left);
        if (live) {
            // [n][r]: row n's chunks in order, chunk p of all at p ^ (n / 8) % 8, so that the lanes of a product,
            // whose rows are 8 apart, find theirs in different banks; [r][n]: rows of 256 bytes
            __syncthreads();                   // (the block before this one has been read)
            for (int p = tid; p < 128 * ranks; p += kThreads) {
                if (TR) {
                    const int r = p >> 4, at = 128 * b + 8 * (p & 15);
                    shared[p] = load8(w + (int64_t)r * a.N + at, a.N - at);
                } else {
                    const int row = p / ranks;
                    v4i v{0, 0, 0, 0};
                    if (128 * b + row < a.N)
                        v = load8(w + (int64_t)128 * b * a.R + 8 * p);
                    shared[p ^ ((row >> 3) & 7)] = v;
                }
            }
            __syncthreads();
            v4f acc[8] = {};
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int c = 4 * g + q;
                const bool there = c < ranks;
                v4i r[8], f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    r[j] = v4i{0, 0, 0, 0};
                    if (there)
                        r[j] = TR ? shared[(8 * c + j) * 16 + i] : shared[((8 * i + j) * ranks + c) ^ (i & 7)];
                }
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    f[m] = r[m];
                    if (TR)                    // eight ranks of eight n: a column for each product
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            f[m][j] = (int)__builtin_amdgcn_perm((uint32_t)r[2 * j + 1][m / 2], (uint32_t)r[2 * j][m / 2],
                                                                 m % 2 ? 0x07060302u : 0x05040100u);
                }
#pragma unroll
                for (int m = 0; m < 8; ++m)
#pragma unroll
                    for (int h = 0; h < kPieces; ++h) acc[m] = mma(v[h][g], f[m], acc[m]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t d = (uint32_t)o[c][e];
                    o[c][e] = pack2(__uint_as_float(d << 16) + acc[2 * e][c],
                                    __uint_as_float(d & 0xFFFF0000u) + acc[2 * e + 1][c]);
                }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (token[c] >= 0)
                store8(a.out + token[c] * a.ldo + n, o[c], left);
    }
}

// ---------------------------------------------------------------------------
// Outer: out[l][r][c] (or [l][c][r]) = sum over the adapter's places of f[r][place] z[token][c].  A wave takes
// 128 columns and 16 RB ranks, 32 places at a time: a lane loads 8 columns of 8 tokens and pairs them up for the
// matrix cores, whose m-th product has the columns 8 i + m.  Waves and splits share the places.  Lines asked of the
// L2 bound it, z's and the factors': 8192 tokens of 5120 and 10240, 16 ranks, 252 MB of z, 69 us (eight waves a
// workgroup 71); of 5120 and 5120, 64 ranks 77 us (135 with 32 ranks at a time, which reads z twice).
// ---------------------------------------------------------------------------
struct OuterJob {
    const uint16_t *z, *pieces;
    float *out;                // [splits] of the result
    int64_t ldz, size;         // size: elements of the result
    int C, blocks, splits;
    int rank_last;             // the result is [l][c][r]
};

struct OuterArgs {
    OuterJob job[2];
    const int32_t *order, *offsets;
    int R, Rp, groups, first;  // workgroups of the first job
};

constexpr int kOuterWaves = 4, kOuterAlone = 64;

template <int RB>
__global__ void __launch_bounds__(64 * kOuterWaves, 2) k_outer(OuterArgs a)
{
    extern __shared__ v4f sums[];              // [waves / 2][RB * 8][64]
    const int second = (int)blockIdx.x >= a.first;
    const OuterJob &job = a.job[second];
    int b = (int)blockIdx.x - (second ? a.first : 0);
    const int split = b % job.splits;
    b /= job.splits;
    const int group = b % a.groups;
    b /= a.groups;
    const int c0 = b % job.blocks * 128, l = b / job.blocks;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    const int beg = a.offsets[l], end = a.offsets[l + 1], r0 = group * 16 * RB;
    // few places: one wave, and no sums of others (1024 tokens of 64 adapters of 16 ranks, K = N = 4096, all kernels: 43 us,
    // four waves 50; with 96 places too 4096 tokens of 51 adapters 89, four waves 88)
    const bool alone = end - beg <= kOuterAlone;
    const int waves = alone ? 1 : kOuterWaves;
    if (alone && wave > 0)
        return;
    const int left = job.C - (c0 + 8 * i);
    const uint16_t *z = job.z + c0 + 8 * i;
    // the pieces of eight places lie together: sixteen lanes load 256 bytes of them (ranks apart by all places
    // fell on few channels of the L2: 85 us for the gradients of 8192 tokens of 5120 and 10240)
    const uint16_t *pieces = job.pieces + (piece_place(beg, l) / 8 + q) * 24 * a.Rp + (r0 + i) * 8;
    v4f acc[RB][8] = {};
    for (int t = beg + 32 * (split * waves + wave); t < end; t += 32 * waves * job.splits) {
        const int first = t + 8 * q, n = end - first;          // this lane's places
        v4i row[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            row[j] = v4i{0, 0, 0, 0};
            if (j < n)
                row[j] = load8(z + a.order[first + j] * job.ldz, left);
        }
        v4i f[3][RB];
#pragma unroll
        for (int h = 0; h < 3; ++h)
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                f[h][r] = v4i{0, 0, 0, 0};
                if (n > 0)
                    f[h][r] = load8(pieces + (t - beg) * 3 * (int64_t)a.Rp + (h * a.Rp + 16 * r) * 8);
            }
        v4i col[8];
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                col[m][j] = (int)__builtin_amdgcn_perm((uint32_t)row[2 * j + 1][m / 2], (uint32_t)row[2 * j][m / 2],
                                                       m % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
        for (int h = 0; h < 3; ++h)
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int m = 0; m < 8; ++m) acc[r][m] = mma(f[h][r], col[m], acc[r][m]);
    }
    for (int half = waves / 2; half > 0; half /= 2) {
        if (wave >= half && wave < 2 * half)
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int m = 0; m < 8; ++m) sums[((wave - half) * RB * 8 + r * 8 + m) * 64 + lane] = acc[r][m];
        __syncthreads();
        if (wave < half)
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int m = 0; m < 8; ++m) acc[r][m] += sums[(wave * RB * 8 + r * 8 + m) * 64 + lane];
        __syncthreads();
    }
    if (wave > 0)
        return;
    float *out = job.out + split * job.size;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        const int rank = r0 + 16 * r + 4 * q;
        if (rank >= a.R)
            continue;
        if (job.rank_last) {
#pragma unroll
            for (int m = 0; m < 8; ++m)
                if (m < left)
                    __builtin_memcpy(out + ((int64_t)l * job.C + c0 + 8 * i + m) * a.R + rank, &acc[r][m], 16);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float *o = out + ((int64_t)l * a.R + rank + c) * job.C + c0 + 8 * i;
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

// out = the splits' parts, added in order, four elements a thread (whole numbers of four: ranks are).  Both gradients in one
// launch: 2048 tokens of an adapter, 16 ranks, K = N = 2048, all kernels 35 us, in two launches 38.
struct AddArgs {
    float *out[2];
    const float *part[2];
    int64_t size[2], first;    // elements; threads of the first gradient
    int splits[2];
};

__global__ void __launch_bounds__(kThreads) k_add_parts(AddArgs a)
{
    const int64_t step = (int64_t)gridDim.x * kThreads, all = a.first + a.size[1] / 4;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += step) {
        const int j = i >= a.first;
        const int64_t at = 4 * (j ? i - a.first : i);
        v4f v = {};
        for (int k = 0; k < a.splits[j]; ++k) {
            v4f t;
            __builtin_memcpy(&t, a.part[j] + k * a.size[j] + at, 16);
            v += t;
        }
        __builtin_memcpy(a.out[j] + at, &v, 16);
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
struct Sizes {
    int64_t T, K, N, R, L;
    int64_t Rp;                // ranks in whole blocks of 16: 1, 2, 4 or 8
    int tb, rb, groups;        // shrink: blocks of tokens and ranks of a workgroup, groups of ranks
    int wide;                  // expand: blocks of tokens
    int max_tiles, max_wides;  // the latter 0 where every tile begins an expand tile
    int splits;                // shrink of the forward call: parts of K
};

// Parts of K that the expand kernel adds: 32 tokens of 28 adapters, K = 5120, N = 10240, both kernels: one part
// 16.3 us, four 13.4, eight 14.6; 164 workgroups (24 adapters of 64 ranks, N = 51200): one 52.9, three 54.6.
constexpr int64_t kMaxSplits = 4;

// Tokens an adapter has on average from which 64 share a load of the expand kernel's weights, not 16 (both kernels): 32
// adapters of 16 ranks, K = N = 5120, of 32 tokens 22.8 us with 64 at a time, 22.4 with 16; 16 adapters of 64 tokens 19.8 and
// 21.8; 32 adapters of 48 tokens, K = N = 2048, 16 ranks 17.8 and 17.5, 64 ranks 23.6 and 25.0.  Up to kWaveTokens tokens never
// (64 of an adapter 12.8 and 12.2).
constexpr int64_t kManyTokens = 40;

Sizes sizes(int64_t T, int64_t K, int64_t N, int64_t R, int64_t L)
{
    Sizes z{T, K, N, R, L, 16, 1, 1, 1, 1, 0, 0, 1};
    while (z.Rp < R) z.Rp *= 2;
    const int64_t mean = T / std::min(L, std::max<int64_t>(T, 1));
    z.wide = mean >= kManyTokens && T > kWaveTokens ? kWide / 16 : 1;
    // shrink: more tokens a workgroup only where there are workgroups for all CUs (both kernels: 8192 tokens of 8
    // adapters of 64 ranks, K = N = 5120, 16 at a time 131 us, 32 116; 131072 of 2 adapters of 16 ranks, K = N = 1024,
    // 16 at a time 274, 32 218, 64 199; 65536 of 64 adapters, K = N = 2048, 189, 187 and 195)
    while (z.tb < z.wide && T >= 16 * 2 * z.tb * 240) z.tb *= 2;
    z.max_tiles = (int)std::max<int64_t>(1, T / (16 * z.tb) + std::min(L + 1, T));
    if (z.wide > z.tb)
        z.max_wides = (int)(T / (16 * z.wide) + std::min(L + 1, T));
    // and 32 ranks a workgroup likewise (64 ranks, K = N = 5120, both kernels: 8192 tokens of 8 adapters, 528 workgroups
    // then, 116 us, 16 at a time 138; 1024 of 32, 194, 36 and 40; 256 of 64, 162, 29 and 27)
    if (z.Rp > 16 && z.max_tiles * (z.Rp / 16) > 360)
        z.rb = 2;
    z.groups = (int)((R + 16 * z.rb - 1) / (16 * z.rb));
    // few workgroups: parts of K, a step for each wave at least (a CU alone loads some 50 GB/s: 256 tokens of an
    // adapter of 16 ranks, K = N = 5120, both kernels: one part 15.2 us, four 12.1)
    if (z.max_tiles * z.groups <= 128)
        z.splits = (int)std::min<int64_t>((K + 8 * kStep - 1) / (8 * kStep), kMaxSplits);
    return z;
}

int outer_blocks(const Sizes &z) { return z.Rp > 32 ? 4 : z.Rp > 16 ? 2 : 1; }

// Splits of the places: both gradients' workgroups fill the CUs once, four to a CU with 16 ranks a workgroup and two with
// more (8192 tokens of an adapter of 16 ranks, K = N = 5120: once 144 us, half of that 161; two of 64 ranks: once 232,
// twice 247).
int outer_splits(const Sizes &z, int64_t C)
{
    const int64_t wgs = z.L * ((C + 127) / 128) * ((z.R + 63) / 64), room = outer_blocks(z) == 1 ? 512 : 256;
    return (int)std::max<int64_t>(1, std::min<int64_t>({room / wgs, z.T / (64 * kOuterWaves), 16}));
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

struct Space {
    int32_t *order, *offsets, *counts;
    int4 *tiles, *wides;
    float *sums;               // the parts of v (backward: u) for expand
    uint16_t *fv, *fu;         // backward: the pieces of s v and s u for outer
    float *outer_a, *outer_b;  // and the parts of dA and dB
    size_t bytes;
};

int plan_digits(int64_t L)
{
    int d = 1;
    while (d <= L) d *= 2;
    return d;
}

Space space(const Sizes &z, void *ws, bool back)
{
    Layout l{static_cast<uint8_t *>(ws)};
    Space f{};
    f.order = l.take<int32_t>(z.T);
    f.tiles = l.take<int4>(z.max_tiles);
    f.wides = z.max_wides ? l.take<int4>(z.max_wides) : nullptr;
    f.counts = l.take<int32_t>(z.T > kSelfTokens ? (int64_t)sort_parts(z.T) * plan_digits(z.L) : 0);
    f.sums = l.take<float>((back ? 1 : z.splits) * z.T * z.Rp);
    if (back) {
        f.offsets = l.take<int32_t>(z.L + 1);
        const int64_t places = piece_place(z.T, (int)z.L);
        f.fv = l.take<uint16_t>(kPieces * z.Rp * places);
        f.fu = l.take<uint16_t>(kPieces * z.Rp * places);
        const int64_t sa = outer_splits(z, z.K), sb = outer_splits(z, z.N);
        f.outer_a = l.take<float>(sa > 1 ? sa * z.L * z.R * z.K : 0);
        f.outer_b = l.take<float>(sb > 1 ? sb * z.L * z.R * z.N : 0);
    }
    f.bytes = l.bytes;
    return f;
}

bool good_shape(int64_t T, int64_t K, int64_t N, int64_t R, int64_t L)
{
    return T >= 0 && T <= kMaxTokens && K > 0 && K <= kMaxWidth && N >= 0 && N <= kMaxWidth && R > 0 && R <= kMaxRank &&
           R % 8 == 0 && L > 0 && L <= kMaxAdapters && L * std::max<int64_t>(R, 64) * std::max(K, N) < (int64_t)1 << 33;
}

Region rows_of(const uint16_t *p, int64_t rows, int64_t width, int64_t ld) { return Region{p, rows, 2 * width, 2 * ld}; }

template <bool BACK>
hipError_t launch_shrink(const Sizes &z, const ShrinkArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)(z.max_tiles * z.groups * (BACK ? 2 : a.splits))), block(64 * kShrinkWaves);
    const size_t lds = std::max(kShrinkWaves * shrink_share(z.tb, z.rb) * sizeof(v4i),
                                a.self == 2 ? kShrinkWaves * (z.L + 1) * sizeof(int32_t) : 0);
    switch (z.rb * 8 + z.tb) {
    case 8 + 1: hipLaunchKernelGGL((k_shrink<1, 1, BACK>), grid, block, lds, s, a); break;
    case 8 + 2: hipLaunchKernelGGL((k_shrink<2, 1, BACK>), grid, block, lds, s, a); break;
    case 8 + 4: hipLaunchKernelGGL((k_shrink<4, 1, BACK>), grid, block, lds, s, a); break;
    case 16 + 1: hipLaunchKernelGGL((k_shrink<1, 2, BACK>), grid, block, lds, s, a); break;
    case 16 + 2: hipLaunchKernelGGL((k_shrink<2, 2, BACK>), grid, block, lds, s, a); break;
    default: hipLaunchKernelGGL((k_shrink<4, 2, BACK>), grid, block, lds, s, a); break;
    }
    return hipGetLastError();
}

// Fills in the plan, and makes it in a launch of its own where the tokens are too many for each workgroup.
hipError_t make_plan(const Sizes &z, const Space &f, const void *ids, int32_t id_bits, ShrinkArgs &a, hipStream_t s)
{
    a.plan = Plan{ids, f.order, f.offsets, f.tiles, f.wides, (int)z.T, (int)z.L, 16 * z.tb, 16 * z.wide, z.max_tiles, z.max_wides, id_bits};
    a.self = z.T == 0 || z.T > kSelfTokens ? 0 : z.T <= kWaveTokens ? 1 : 2;
    if (a.self)
        return hipSuccess;
    const int blocks = std::max(1, sort_parts(z.T));
    const ManyArgs m{a.plan, SortRange{(int)z.T, sort_share(z.T, blocks), blocks, z.T > kSelfTokens ? f.counts : nullptr},
                     plan_digits(z.L)};
    if (m.range.counts) {
        hipLaunchKernelGGL(k_plan_count, dim3(blocks), dim3(kSortThreads), m.digits * sizeof(int32_t), s, m);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(k_plan_place, dim3(blocks), dim3(kSortThreads), place_lds(m.digits), s, m);
    return hipGetLastError();
}

template <int G, bool TR>
void expand_kernel(const Sizes &z, const ExpandArgs &a, dim3 grid, hipStream_t s)
{
    if (z.wide > 1)
        hipLaunchKernelGGL((k_expand_many<G, TR>), grid, dim3(kThreads), 128 * 2 * (size_t)z.R, s, a);
    else
        hipLaunchKernelGGL((k_expand_few<G, TR>), grid, dim3(kThreads), 0, s, a);
}

template <bool TR>
hipError_t launch_expand(const Sizes &z, const Space &f, const float *scale, const uint16_t *w, int64_t N, const uint16_t *base, int64_t ldb,
                         uint16_t *out, int64_t ldo, hipStream_t s)
{
    // Workgroups of a tile.  Many tokens: three blocks of 128 n each at most (65536 tokens, K = N = 2048, 16 ranks, both
    // kernels: one block 193 us, three 187, four 202, eight 221; 8192 tokens, 5120 and 5120, 64 ranks: one 118, three 116),
    // fewer where the tiles alone are too few
    const int64_t full = z.wide > 1 ? (N + 127) / 128 : (N + 64 * kWaves - 1) / (64 * kWaves);
    const int64_t tiles = z.max_wides ? z.max_wides : z.max_tiles, least = z.wide > 1 ? (full + 2) / 3 : 1;
    const int64_t want = std::max(least, std::min<int64_t>(full, (z.wide > 1 ? 2048 : 8192) / tiles));
    const int chunks = (int)std::max<int64_t>(1, std::min<int64_t>(want, (((int64_t)1 << 24) - 1) / tiles));
    const ExpandArgs a{f.sums, scale, (int)z.T, TR ? 1 : z.splits, f.order, f.wides ? f.wides : f.tiles, w, base, out, ldb, ldo, (int)N, (int)z.R, (int)z.Rp, chunks};
    const dim3 grid((unsigned)(tiles * chunks));
    if (z.R <= 32)
        expand_kernel<1, TR>(z, a, grid, s);
    else if (z.R <= 64)
        expand_kernel<2, TR>(z, a, grid, s);
    else
        expand_kernel<4, TR>(z, a, grid, s);
    return hipGetLastError();
}

// Workgroups of the kernel that has both products: 512 n of a tile each.
int64_t both_chunks(int64_t N) { return (N + 64 * kShrinkWaves - 1) / (64 * kShrinkWaves); }

// Whether it is taken (16 ranks, both kernels): K = 2048, 16 tokens of 12 adapters on N = 10240, some 240 workgroups, 8.5
// us, in two launches 9.6; 32 of 28, 560 workgroups, 19.8 and 12.2; a token, K = N = 4096 7.5 and 7.5, 5120 8.5 and 7.9.
bool one_launch(const Sizes &z)
{
    return z.T <= kWaveTokens && z.wide == 1 && z.Rp <= 32 && z.Rp * z.K <= 65536 && z.max_tiles * both_chunks(z.N) <= 320;   // (with tiles that stay empty)
}

hipError_t launch_both(const Sizes &z, const Space &f, const void *ids, int32_t id_bits, ShrinkArgs &a, const float *scale,
                       const uint16_t *w, const uint16_t *base, int64_t ldb, uint16_t *out, int64_t ldo, hipStream_t s)
{
    const hipError_t p = make_plan(z, f, ids, id_bits, a, s);          // (no launch: every wave makes its own)
    if (p != hipSuccess)
        return p;
    const int chunks = (int)both_chunks(z.N);
    const ExpandArgs e{nullptr, scale, (int)z.T, 1, nullptr, nullptr, w, base, out, ldb, ldo, (int)z.N, (int)z.R, (int)z.Rp, chunks};
    const dim3 grid((unsigned)(z.max_tiles * chunks)), block(64 * kShrinkWaves);
    const size_t lds = kShrinkWaves * shrink_share(1, (int)z.Rp / 16) * sizeof(v4i);
    if (z.Rp == 16)
        hipLaunchKernelGGL((k_both<1>), grid, block, lds, s, a, e);
    else
        hipLaunchKernelGGL((k_both<2>), grid, block, lds, s, a, e);
    return hipGetLastError();
}

hipError_t launch_outer(const Sizes &z, const Space &f, const uint16_t *x, int64_t ldx, const uint16_t *dy, int64_t lddy,
                        float *da, float *db, hipStream_t s)
{
    const int sa = outer_splits(z, z.K), sb = outer_splits(z, z.N), rb = outer_blocks(z);
    OuterArgs a{};
    a.job[0] = OuterJob{x, f.fu, sa > 1 ? f.outer_a : da, ldx, z.L * z.R * z.K, (int)z.K, (int)((z.K + 127) / 128), sa, 0};
    a.job[1] = OuterJob{dy, f.fv, sb > 1 ? f.outer_b : db, lddy, z.L * z.R * z.N, (int)z.N, (int)((z.N + 127) / 128), sb, 1};
    a.order = f.order;
    a.offsets = f.offsets;
    a.R = (int)z.R;
    a.Rp = (int)z.Rp;
    a.groups = (int)((z.R + 16 * rb - 1) / (16 * rb));
    a.first = (int)(z.L * a.job[0].blocks * a.groups * sa);
    const dim3 grid((unsigned)(a.first + z.L * a.job[1].blocks * a.groups * sb)), block(64 * kOuterWaves);
    const size_t lds = (size_t)kOuterWaves / 2 * rb * 8 * 64 * sizeof(v4f);
    if (rb == 1)
        hipLaunchKernelGGL((k_outer<1>), grid, block, lds, s, a);
    else if (rb == 2)
        hipLaunchKernelGGL((k_outer<2>), grid, block, lds, s, a);
    else
        hipLaunchKernelGGL((k_outer<4>), grid, block, lds, s, a);
    const hipError_t e = hipGetLastError();
    AddArgs add{};
    for (int j = 0; j < 2; ++j) {
        const OuterJob &o = a.job[j];
        add.out[j] = j ? db : da;
        add.part[j] = o.out;
        add.size[j] = o.splits > 1 ? o.size : 0;
        add.splits[j] = o.splits;
    }
    add.first = add.size[0] / 4;
    const int64_t blocks = (add.first + add.size[1] / 4 + kThreads - 1) / kThreads;
    if (e != hipSuccess || blocks == 0)
        return e;
    hipLaunchKernelGGL(k_add_parts, dim3((unsigned)std::min<int64_t>(blocks, 4096)), dim3(kThreads), 0, s, add);
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
    return space(sizes(tokens, K, N, rank, adapters), nullptr, false).bytes;
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
    const Space f = space(z, workspace, false);
    if (!workspace || workspace_bytes < f.bytes)
        return QLIN_ERR_WORKSPACE;
    const Region x = rows_of(X, tokens, K, ldx), y = rows_of(Y, tokens, N, ldy), add = rows_of(base, tokens, N, ldb),
                 fa = flat(A, 2 * adapters * rank * K), fb = flat(B, 2 * adapters * N * rank),
                 id = flat(ids, tokens * (id_bits / 8)), sc = flat(scale, 4 * adapters);
    if (overlaps({y, flat(workspace, f.bytes)}, {x, fa, fb, id, sc, same(y, add) ? Region{} : add}))
        return QLIN_ERR_BAD_ARGUMENT;
    hipStream_t s = static_cast<hipStream_t>(stream);
    ShrinkArgs a{};
    a.job[0] = ShrinkJob{X, A, f.sums, nullptr, ldx, (int)K};
    a.splits = z.splits;
    a.scale = scale;
    a.R = (int)rank;
    a.Rp = (int)z.Rp;
    a.groups = z.groups;
    if (one_launch(z))
        return launch_both(z, f, ids, id_bits, a, scale, B, base, ldb, Y, ldy, s) == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
    if (make_plan(z, f, ids, id_bits, a, s) != hipSuccess || launch_shrink<false>(z, a, s) != hipSuccess ||
        launch_expand<false>(z, f, scale, B, N, base, ldb, Y, ldy, s) != hipSuccess)
        return QLIN_ERR_HIP;
    return QLIN_OK;
}

size_t qlin_lora_backward_workspace_size(int64_t tokens, int64_t K, int64_t N, int64_t rank, int64_t adapters)
{
    if (!good_shape(tokens, K, N, rank, adapters) || N == 0)
        return 0;
    return space(sizes(tokens, K, N, rank, adapters), nullptr, true).bytes;
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
    const Space f = space(z, workspace, true);
    if (!workspace || workspace_bytes < f.bytes)
        return QLIN_ERR_WORKSPACE;
    const Region x = rows_of(X, tokens, K, ldx), dy = rows_of(dY, tokens, N, lddy), dx = rows_of(dX, tokens, K, lddx),
                 add = rows_of(base, tokens, K, ldb), fa = flat(A, 2 * adapters * rank * K),
                 fb = flat(B, 2 * adapters * N * rank), id = flat(ids, tokens * (id_bits / 8)), sc = flat(scale, 4 * adapters);
    const bool in_place = tokens > 0 && same(dx, add);
    if (overlaps({dx, flat(dA, 4 * adapters * rank * K), flat(dB, 4 * adapters * N * rank), flat(workspace, f.bytes)},
                 {x, dy, fa, fb, id, sc, in_place ? Region{} : add}))
        return QLIN_ERR_BAD_ARGUMENT;
    hipStream_t s = static_cast<hipStream_t>(stream);
    ShrinkArgs a{};
    a.job[0] = ShrinkJob{X, A, nullptr, f.fv, ldx, (int)K};
    a.job[1] = ShrinkJob{dY, B, f.sums, f.fu, lddy, (int)N};
    a.splits = 1;
    a.scale = scale;
    a.R = (int)rank;
    a.Rp = (int)z.Rp;
    a.groups = z.groups;
    if (make_plan(z, f, ids, id_bits, a, s) != hipSuccess)
        return QLIN_ERR_HIP;
    if (tokens > 0 && (launch_shrink<true>(z, a, s) != hipSuccess ||
                       launch_expand<true>(z, f, scale, A, K, base, ldb, dX, lddx, s) != hipSuccess))
        return QLIN_ERR_HIP;
    if (launch_outer(z, f, X, ldx, dY, lddy, dA, dB, s) != hipSuccess)
        return QLIN_ERR_HIP;
    return QLIN_OK;
}

}  // extern "C"
