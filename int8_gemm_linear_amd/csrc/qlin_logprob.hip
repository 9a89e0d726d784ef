// Log probabilities of given tokens, with the entropy of each row, its best
// alternatives, and the gradient of both with respect to the logits.
//
// For a row x of V logits, m = max x, S = sum e^(x - m), W = sum e^(x - m) (x - m):
//   lse = m + ln S,   log p_v = (x_v - m) - ln S,   H = ln S - W / S,
//   dx_v = g ([v = target] - p_v) - h p_v (log p_v + H)
// with g and h the gradients of the target's log p and of H.  One pass over the
// logits keeps m, S, W and the best alternatives; a lane rescales its own S and W
// when its maximum rises: from m to n, W becomes (W + S (m - n)) e^(m - n).
//
// x - m is taken before the product with log2 e, so that rows far from zero lose
// nothing in p and H (lse itself is rounded to fp32), and below -200 it counts as
// -200 where it is multiplied with e^(x - m), which is 0 there: banned tokens (-inf,
// or a type's lowest value) add 0.  The gradient has only the rounded lse to take p
// from, so its p are off by |lse| 2^-24 relatively.
#include <algorithm>
#include <float.h>

#include "qlin_dpp.h"
#include "qlin_elem.h"
#include "qlin_overlap.h"
#include "qlinear.h"

namespace qlin {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPieces = 4;                     // 16-byte pieces a thread takes at a time (two: 113 us where four take 105)
constexpr int kMaxTop = 64;                    // an alternative for each lane of a wave
constexpr int kMaxParts = 64;                  // a part for each lane of the joining wave
// Workgroups that fewer rows are divided into: five run on a CU at once (48 rows of 100003, 5 alternatives: 13.9 us,
// with 2048 workgroups 15.4; 512 rows of 131072, 20 alternatives 50.6 and 56).
constexpr int64_t kRowBlocks = 1280;
constexpr int64_t kMaxRows = (int64_t)1 << 23; // one part each: below 2^32 threads
constexpr int64_t kMaxVocab = (int64_t)1 << 28;
constexpr int64_t kMaxStride = (int64_t)1 << 31;
constexpr float kLowest = -200.0f, kLog2e = 1.4426950408889634f;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

__device__ inline float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

// m, S and W of a part of a row (or of a lane's share of it).
struct Stat {
    float m, s, w;
};

__device__ inline void rescale(Stat &a, float m)
{
    const float r = fmaxf(a.m - m, kLowest), f = exp_of(r);
    a.w = (a.w + a.s * r) * f;
    a.s *= f;
    a.m = m;
}

// An alternative as one number that orders by value, then by the lower index;
// 0 is none, and so are NaNs.
__device__ inline uint64_t key_of(float v, int at)
{
    const int b = __float_as_int(v + 0.0f);                  // -0 and +0 are equal
    const uint32_t o = b < 0 ? ~(uint32_t)b : (uint32_t)b | 0x80000000u;
    return v == v ? (uint64_t)o << 32 | (0xFFFFFFFFu - (uint32_t)at) : 0;
}

__device__ inline float key_value(uint64_t k)
{
    const uint32_t o = (uint32_t)(k >> 32);
    return k == 0 ? __int_as_float(0x7FC00000) : __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

__device__ inline int key_index(uint64_t k) { return k == 0 ? -1 : (int)(0xFFFFFFFFu - (uint32_t)k); }

__device__ inline uint64_t key_lane(uint64_t k, int lane)
{
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)k, lane);
}

// A wave's best `top` keys so far, in order, one a lane.
struct Best {
    uint64_t mine = 0, last = 0;               // this lane's; that of lane top - 1
    float bar = -INFINITY;                     // last's value: a greater one enters

    // A key above `last` (the same in all lanes) goes to its place, the lower ones one lane on.
    __device__ void insert(uint64_t k, int lane, int top)
    {
        const int at = __popcll(__ballot(mine > k));
        const uint64_t up = (uint64_t)(uint32_t)__builtin_amdgcn_update_dpp(0, (int)(mine >> 32), 0x138, 0xF, 0xF, false) << 32 |
                            (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mine, 0x138, 0xF, 0xF, false);   // wave_shr:1
        mine = lane < at ? mine : lane == at ? k : up;
        last = key_lane(mine, top - 1);
    }
};

// A value that at least `top` lanes' v reach: the upper 16 bits, bit by bit, of the top-th greatest.
__device__ inline float top_th(float v, int top)
{
    const int b = __float_as_int(v + 0.0f);
    const uint32_t o = (b < 0 ? ~(uint32_t)b : (uint32_t)b | 0x80000000u) >> 16;
    uint32_t t = 0;
#pragma unroll
    for (int i = 15; i >= 0; --i) {
        const uint32_t more = t | 1u << i;
        t = __popcll(__ballot(o >= more)) >= top ? more : t;
    }
    t <<= 16;
    return t < 0x00800000u ? -INFINITY : __uint_as_float(t & 0x80000000u ? t & 0x7FFFFFFFu : ~t);
}

struct Args {
    const uint8_t *x;
    int64_t ld, ldo;                           // bytes
    const void *target;
    float *logprob, *entropy, *lse, *top_v;
    int32_t *top_id;
    float *stat;                               // [rows][parts][4]: m, S, W, unused
    uint64_t *list;                            // [rows][parts][top]
    const float *g, *h, *lse_in, *entropy_in;  // gradient
    uint8_t *out;
    int V, top, parts, per, id_bits;
};

__device__ inline int target_of(const Args &a, int64_t row)
{
    const int64_t t = a.id_bits == 64 ? static_cast<const int64_t *>(a.target)[row] : static_cast<const int32_t *>(a.target)[row];
    return t >= 0 && t < a.V ? (int)t : -1;
}

// The logit of the row's target, 0 for none: loaded first, used last.
template <typename T>
__device__ inline float target_logit(const Args &a, int64_t row, int target)
{
    return target >= 0 ? Elem<T>::get(reinterpret_cast<const T *>(a.x + row * a.ld)[target]) : 0.0f;
}

// The row's outputs from its statistics; the keys are in `best`.  A row that
// holds no number above -inf has no distribution: log probabilities -inf, H = 0.
__device__ inline void finish(const Args &a, int64_t row, Stat s, const uint64_t *best, int tid, int target, float x)
{
    const float ln = logf(s.s);
    const bool none = s.s == 0.0f;
    if (tid == 0) {
        a.logprob[row] = target < 0 ? 0.0f : none ? -INFINITY : (x - s.m) - ln;
        a.entropy[row] = none ? 0.0f : ln - s.w / s.s;
        a.lse[row] = none ? -INFINITY : s.m + ln;
    }
    if (tid < a.top) {
        const uint64_t k = best[tid];
        a.top_v[row * a.top + tid] = k == 0 ? key_value(k) : none ? -INFINITY : (key_value(k) - s.m) - ln;
        a.top_id[row * a.top + tid] = key_index(k);
    }
}

// The pieces of chunk c, values behind `end` as -inf.
template <typename T>
__device__ inline void load_chunk(v4i (&p)[kPieces], const T *x, int c, int end, int tid)
{
    constexpr int E = 16 / sizeof(T);
    if (c + kThreads * E * kPieces <= end) {
#pragma unroll
        for (int u = 0; u < kPieces; ++u) p[u] = load_piece(x + c + (u * kThreads + tid) * E);
        return;
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
        const int at = c + (u * kThreads + tid) * E;
        if (at + E <= end) {
            p[u] = load_piece(x + at);
        } else {
            T t[E];
#pragma unroll
            for (int i = 0; i < E; ++i) t[i] = at + i < end ? x[at + i] : Elem<T>::put(-INFINITY);
            __builtin_memcpy(&p[u], t, 16);
        }
    }
}

// A part of a row for each workgroup, a chunk's loads on their way while the one before is added up.  The logits'
// bytes bound it, with the exponentials close behind (the vector units are busy for five sixths of the time): 2047
// rows of 131072 in bf16, 98 us, 5.5 TB/s, with one alternative 105 us.
template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads) k_logprobs(Args a)
{
    constexpr int E = 16 / sizeof(T), kStep = kThreads * E * kPieces;
    __shared__ uint64_t keys[TOP ? kWaves : 1][kMaxTop], merged[kMaxTop];
    __shared__ Stat stats[kWaves];
    // For each wave a value that a quarter of `top` of its logits reach: the least of them bounds what can be among
    // the alternatives (2047 rows of 131072, 20 alternatives: 122 us, with each wave's own list alone 146)
    __shared__ float reached[kWaves];
    const int quarter = (a.top + kWaves - 1) / kWaves;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x / a.parts;
    const int part = blockIdx.x % a.parts, beg = part * a.per, end = min(beg + a.per, a.V);
    const T *x = reinterpret_cast<const T *>(a.x + row * a.ld);
    const int target = a.parts == 1 ? target_of(a, row) : -1;
    const float logit = target_logit<T>(a, row, target);
    Stat s{-FLT_MAX, 0.0f, 0.0f};
    Best best;
    v4i next[kPieces];
    load_chunk(next, x, beg, end, tid);
    for (int c = beg; c < end; c += kStep) {
        float v[kPieces][E], high[kPieces], most = -INFINITY;
        const int pieces = min(kPieces, (end - c + kThreads * E - 1) / (kThreads * E));    // that hold anything
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            if (u >= pieces)
                break;
            piece_values<T>(v[u], next[u]);
            high[u] = v[u][0];
#pragma unroll
            for (int i = 1; i < E; ++i) high[u] = fmaxf(high[u], v[u][i]);
            most = fmaxf(most, high[u]);
        }
        if (c + kStep < end)
            load_chunk(next, x, c + kStep, end, tid);
        if (most > s.m)
            rescale(s, most);
        // (a turn's terms join the others as one sum: each by itself, next to a term of 1, those below 2^-24 were lost)
        float turn_s = 0.0f, turn_w = 0.0f;
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            if (u >= pieces)
                break;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float d = v[u][i] - s.m, e = exp_of(d);
                turn_s += e;
                turn_w = fmaf(e, fmaxf(d, kLowest), turn_w);
            }
        }
        s.s += turn_s;
        s.w += turn_w;
        if (TOP) {
            // Of the first chunk, the lanes' maxima give the bound; later, a value also has to be greater than the
            // last of the wave's list, whose index is lower.
            if (c == beg) {
                const float r = top_th(most, quarter);
                if (lane == 0)
                    reached[wave] = r;
                __syncthreads();
            }
            float bound = INFINITY;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) bound = fminf(bound, const_cast<volatile float *>(reached)[w]);
            const float bar = best.bar;
            const bool open = best.last == 0;
            bool entered = false;
#pragma unroll
            for (int u = 0; u < kPieces; ++u) {
                if (u >= pieces)
                    break;
                if (!__ballot(high[u] >= bound && (open || high[u] > bar)))
                    continue;
                const int at = c + (u * kThreads + tid) * E;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const uint64_t k = at + i < end && v[u][i] >= bound ? key_of(v[u][i], at + i) : 0;
                    uint64_t in = __ballot(k > best.last);
                    while (in) {
                        const uint64_t one = key_lane(k, __ffsll((unsigned long long)in) - 1);
                        best.insert(one, lane, a.top);
                        entered = true;
                        in &= in - 1;
                        in &= __ballot(k > best.last);
                    }
                }
            }
            if (entered) {
                best.bar = best.last ? key_value(best.last) : -INFINITY;
                const uint64_t k = key_lane(best.mine, quarter - 1);
                if (k && lane == 0)
                    const_cast<volatile float *>(reached)[wave] = fmaxf(key_value(k), reached[wave]);
            }
        }
    }
    // one statistic a wave, then one for all
    const float m = wave_max(s.m);
    rescale(s, m);
    s.s = wave_sum(s.s);
    s.w = wave_sum(s.w);
    if (lane == 0)
        stats[wave] = s;
    if (TOP) {
        keys[wave][lane] = lane < a.top ? best.mine : 0;
        if (wave == 0)
            merged[lane] = 0;
    }
    __syncthreads();
    s = stats[0];
    for (int w = 1; w < kWaves; ++w) s.m = fmaxf(s.m, stats[w].m);
    {
        Stat t = stats[0];
        rescale(t, s.m);
        s.s = t.s;
        s.w = t.w;
        for (int w = 1; w < kWaves; ++w) {
            t = stats[w];
            rescale(t, s.m);
            s.s += t.s;
            s.w += t.w;
        }
    }
    if (TOP) {
        if (tid < kWaves * a.top) {
            const uint64_t k = keys[tid / a.top][tid % a.top];
            int rank = 0;
            for (int j = 0; j < a.top; j += 4)
#pragma unroll
                for (int e = 0; e < 4 * kWaves; ++e) rank += keys[e / 4][j + e % 4] > k ? 1 : 0;
            if (k && rank < a.top)
                merged[rank] = k;
        }
        __syncthreads();
    }
    if (a.parts == 1) {
        finish(a, row, s, merged, tid, target, logit);
        return;
    }
    const int64_t p = row * a.parts + part;
    if (tid == 0) {
        a.stat[4 * p] = s.m;
        a.stat[4 * p + 1] = s.s;
        a.stat[4 * p + 2] = s.w;
    }
    if (TOP && tid < a.top)
        a.list[p * a.top + tid] = merged[tid];
}

// The parts of a row, for the few rows of a decoding step (1 row of 131072, 20 alternatives: both kernels 10.4 us, most
// of it their launches and two trips to memory).  A value that `top` of the parts' best reach bounds what can be among the alternatives; what
// reaches it is gathered and ranked.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_logprobs_join(Args a)
{
    constexpr int kHold = 4;                   // keys a thread loads first
    __shared__ uint64_t merged[kMaxTop], kept[kMaxParts * kMaxTop];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row = blockIdx.x, p = row * a.parts + lane;
    const uint64_t *list = a.list + row * a.parts * a.top;
    const int all = a.parts * a.top, target = target_of(a, row);
    Stat s{-FLT_MAX, 0.0f, 0.0f};
    if (lane < a.parts)
        s = Stat{a.stat[4 * p], a.stat[4 * p + 1], a.stat[4 * p + 2]};
    const uint64_t head = a.top && lane < a.parts ? list[lane * a.top] : 0;
    uint64_t mine[kHold];
#pragma unroll
    for (int h = 0; h < kHold; ++h) mine[h] = tid + h * kThreads < all ? list[tid + h * kThreads] : 0;
    const float logit = target_logit<T>(a, row, target);
    if (a.top) {
        if (tid == 0)
            count = 0;
        if (tid < kMaxTop)
            merged[tid] = 0;
        __syncthreads();
        const float bar = top_th(head ? key_value(head) : -INFINITY, a.top);
        const auto keep = [&](uint64_t k) {
            if (k && key_value(k) >= bar)
                kept[atomicAdd(&count, 1)] = k;
        };
#pragma unroll
        for (int h = 0; h < kHold; ++h) keep(mine[h]);
        for (int e = tid + kHold * kThreads; e < all; e += kThreads) keep(list[e]);
        __syncthreads();
        const int n = count;
        for (int e = tid; e < n; e += kThreads) {
            const uint64_t k = kept[e];
            int rank = 0;
#pragma unroll 8
            for (int l = 0; l < n; ++l) rank += kept[l] > k ? 1 : 0;
            if (rank < a.top)
                merged[rank] = k;
        }
        __syncthreads();
    }
    rescale(s, wave_max(s.m));
    s.s = wave_sum(s.s);
    s.w = wave_sum(s.w);
    finish(a, row, s, merged, tid, target, logit);
}

// The logits' gradient: a part of a row for each workgroup, read and written once, which bounds it (4096 rows of 100003
// in bf16, 280 us, 5.8 TB/s).
// A row with g = h = 0 (padding) gets zeros and is not read, one without a distribution zeros.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_logprobs_backward(Args a)
{
    constexpr int E = 16 / sizeof(T), kStep = kThreads * E * kPieces;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / a.parts;
    const int part = blockIdx.x % a.parts, beg = part * a.per, end = min(beg + a.per, a.V);
    const T *x = reinterpret_cast<const T *>(a.x + row * a.ld);
    T *out = reinterpret_cast<T *>(a.out + row * a.ldo);
    const int target = target_of(a, row);
    const float lse = a.lse_in[row], g = target >= 0 ? a.g[row] : 0.0f, h = a.h ? a.h[row] : 0.0f,
                entropy = a.h ? a.entropy_in[row] : 0.0f;
    const bool zero = (g == 0.0f && h == 0.0f) || lse == -INFINITY;
    for (int c = beg; c < end; c += kStep) {
        v4i p[kPieces];
        if (!zero)
            load_chunk(p, x, c, end, tid);
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            const int at = c + (u * kThreads + tid) * E;
            float v[E] = {};
            if (!zero) {
                piece_values<T>(v, p[u]);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float z = v[i] - lse;
                    v[i] = -exp_of(z) * fmaf(h, fmaxf(z, kLowest) + entropy, g);
                    if (at + i == target)
                        v[i] += g;
                }
            }
            if (at + E <= end) {
                const v4i o = value_piece<T>(v);
                __builtin_memcpy(out + at, &o, 16);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i)
                    if (at + i < end)
                        out[at + i] = Elem<T>::put(v[i]);
            }
        }
    }
}

int elem_size(qlin_row_type rt)
{
    return rt == QLIN_ROW_F32 ? 4 : rt == QLIN_ROW_BF16 || rt == QLIN_ROW_F16 ? 2 : 0;
}

// Parts of a row: enough workgroups for the GPU where there are few rows (two parts up to kRowBlocks / 2 rows, more for
// fewer), and no more than whole turns of kPieces leave any work where a part has several: 100 rows of 100003 in fp32, 20
// alternatives, 25.7 us, as many as kRowBlocks allow 27.5; without alternatives 12.7 and 13.7.
int row_parts(int es, int64_t rows, int64_t V)
{
    const int64_t chunk = 16 / es * kThreads, pieces = (V + chunk - 1) / chunk;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(kRowBlocks / std::max<int64_t>(rows, 1), kMaxParts));
    int64_t per = (pieces + want - 1) / want;
    if (per > kPieces)
        per = (per + kPieces - 1) / kPieces * kPieces;
    return (int)((pieces + per - 1) / per);
}

// Elements of each part, whole pieces of a workgroup's threads dealt evenly, and the parts that then have any.  Whole turns
// for all parts but the last would help rows without alternatives (400 rows of 50257 in bf16 17.1 -> 14.9 us) and cost
// those with (20 alternatives 31.4 -> 33.8; 640 rows 38.6 -> 41.3).
void divide(Args &a, int es, int64_t parts)
{
    const int64_t chunk = 16 / es * kThreads, pieces = (a.V + chunk - 1) / chunk, per = (pieces + parts - 1) / parts;
    a.per = (int)std::min<int64_t>(per * chunk, a.V);
    a.parts = (int)((pieces + per - 1) / per);
}

qlin_status check(qlin_row_type rt, int32_t id_bits, int64_t rows, int64_t V, const void *x, int64_t ld,
                  const void *target)
{
    const int es = elem_size(rt);
    if (!es || (id_bits != 32 && id_bits != 64))
        return QLIN_ERR_BAD_ARGUMENT;
    if (rows < 0 || rows > kMaxRows || V <= 0 || V > kMaxVocab)
        return QLIN_ERR_BAD_SHAPE;
    if (rows == 0)
        return QLIN_OK;
    if (!x || !target)
        return QLIN_ERR_NULL_POINTER;
    if (ld < V || ld > kMaxStride)
        return QLIN_ERR_BAD_STRIDE;
    if (!aligned(x, es) || !aligned(target, id_bits / 8))
        return QLIN_ERR_MISALIGNED;
    return QLIN_OK;
}

template <typename T>
hipError_t launch_forward(const Args &a, int64_t rows, hipStream_t s)
{
    const dim3 grid((unsigned)(rows * a.parts));
    if (a.top)
        hipLaunchKernelGGL((k_logprobs<T, true>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((k_logprobs<T, false>), grid, dim3(kThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1)
        return e;
    hipLaunchKernelGGL((k_logprobs_join<T>), dim3((unsigned)rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_backward(const Args &a, int64_t rows, hipStream_t s)
{
    hipLaunchKernelGGL((k_logprobs_backward<T>), dim3((unsigned)(rows * a.parts)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

size_t qlin_token_logprobs_workspace_size(qlin_row_type rt, int64_t rows, int64_t V, int64_t top)
{
    const int es = elem_size(rt);
    if (!es || rows <= 0 || rows > kMaxRows || V <= 0 || V > kMaxVocab || top < 0 || top > kMaxTop)
        return 0;
    const int parts = row_parts(es, rows, V);
    return parts > 1 ? (size_t)rows * parts * (16 + 8 * top) : 0;
}

qlin_status qlin_token_logprobs(qlin_row_type rt, int32_t id_bits, int64_t rows, int64_t V, int64_t top,
                                const void *logits, int64_t ld, const void *target, float *logprob,
                                float *entropy, float *lse, float *top_logprob, int32_t *top_id,
                                void *workspace, size_t workspace_bytes, void *stream)
{
    const qlin_status st = check(rt, id_bits, rows, V, logits, ld, target);
    if (st != QLIN_OK)
        return st;
    if (top < 0 || top > kMaxTop || top > V)
        return QLIN_ERR_BAD_SHAPE;
    if (rows == 0)
        return QLIN_OK;
    if (!logprob || !entropy || !lse || (top > 0 && (!top_logprob || !top_id)))
        return QLIN_ERR_NULL_POINTER;
    if (!aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(lse, 4) || !aligned(top_logprob, 4) ||
        !aligned(top_id, 4) || !aligned(workspace, 8))
        return QLIN_ERR_MISALIGNED;
    const size_t need = qlin_token_logprobs_workspace_size(rt, rows, V, top);
    if (need && (!workspace || workspace_bytes < need))
        return QLIN_ERR_WORKSPACE;
    const int es = elem_size(rt);
    if (overlaps({flat(logprob, 4 * rows), flat(entropy, 4 * rows), flat(lse, 4 * rows), flat(top_logprob, 4 * rows * top),
                  flat(top_id, 4 * rows * top), flat(workspace, need)},
                 {Region{logits, rows, V * es, ld * es}, flat(target, rows * (id_bits / 8))}))
        return QLIN_ERR_BAD_ARGUMENT;
    Args a{};
    a.x = static_cast<const uint8_t *>(logits);
    a.ld = ld * es;
    a.target = target;
    a.logprob = logprob;
    a.entropy = entropy;
    a.lse = lse;
    a.top_v = top_logprob;
    a.top_id = top_id;
    a.V = (int)V;
    a.top = (int)top;
    a.id_bits = id_bits;
    divide(a, es, row_parts(es, rows, V));
    a.list = static_cast<uint64_t *>(workspace);
    a.stat = reinterpret_cast<float *>(a.list + (size_t)rows * a.parts * top);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = rt == QLIN_ROW_F32 ? launch_forward<float>(a, rows, s)
                         : rt == QLIN_ROW_BF16 ? launch_forward<uint16_t>(a, rows, s)
                                               : launch_forward<__half>(a, rows, s);
    return e == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
}

qlin_status qlin_token_logprobs_backward(qlin_row_type rt, int32_t id_bits, int64_t rows, int64_t V,
                                         const float *dlogprob, const float *dentropy, const void *logits,
                                         int64_t ld, const void *target, const float *lse,
                                         const float *entropy, void *dlogits, int64_t ldo, void *stream)
{
    const qlin_status st = check(rt, id_bits, rows, V, logits, ld, target);
    if (st != QLIN_OK || rows == 0)
        return st;
    if (!dlogprob || !lse || !dlogits || (dentropy && !entropy))
        return QLIN_ERR_NULL_POINTER;
    if (ldo < V || ldo > kMaxStride)
        return QLIN_ERR_BAD_STRIDE;
    const int es = elem_size(rt);
    if (!aligned(dlogits, es) || !aligned(dlogprob, 4) || !aligned(dentropy, 4) || !aligned(lse, 4) ||
        !aligned(entropy, 4))
        return QLIN_ERR_MISALIGNED;
    const Region x{logits, rows, V * es, ld * es}, dx{dlogits, rows, V * es, ldo * es};
    if (overlaps({dx}, {same(dx, x) ? Region{} : x, flat(target, rows * (id_bits / 8)), flat(dlogprob, 4 * rows),
                        flat(dentropy, 4 * rows), flat(lse, 4 * rows), flat(dentropy ? entropy : nullptr, 4 * rows)}))
        return QLIN_ERR_BAD_ARGUMENT;
    Args a{};
    a.x = static_cast<const uint8_t *>(logits);
    a.out = static_cast<uint8_t *>(dlogits);
    a.ld = ld * es;
    a.ldo = ldo * es;
    a.target = target;
    a.g = dlogprob;
    a.h = dentropy;
    a.lse_in = lse;
    a.entropy_in = entropy;
    a.V = (int)V;
    a.id_bits = id_bits;
    // a chunk for each workgroup, as far as the rows leave a launch room for them
    const int64_t chunk = 16 / es * kThreads * kPieces, most = (((int64_t)1 << 24) - 1) / rows;
    divide(a, es, std::max<int64_t>(1, std::min((V + chunk - 1) / chunk, most)));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = rt == QLIN_ROW_F32 ? launch_backward<float>(a, rows, s)
                         : rt == QLIN_ROW_BF16 ? launch_backward<uint16_t>(a, rows, s)
                                               : launch_backward<__half>(a, rows, s);
    return e == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
}

}  // extern "C"
