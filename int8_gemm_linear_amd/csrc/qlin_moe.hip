// Routing of tokens to experts around the grouped products: the sort of
// (token, choice) slots by expert, the copies of token rows in that order,
// the weighted return, and the gradients of both directions.
//
// Slot i = token * topk + choice has the expert id topk_ids[i].  With
// c[e] = #{i : id[i] = e},
//   offsets[e] = sum_{e' < e} c[e'],
//   row[i]     = offsets[id[i]] + #{i' < i : id[i'] = id[i]},
// a stable counting sort, so rows do not depend on timing.  Everything else
// is addressed by row[i]: permute scatters token rows to row[i], combine and
// the gradients gather from it.  All of it moves bytes once; HBM bounds the
// long calls and the launch the short ones.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "qlin_device.h"
#include "qlin_dpp.h"
#include "qlin_moe_scan.h"
#include "qlinear.h"

namespace qlin {
namespace {

constexpr int64_t kMaxSlots = ((int64_t)1 << 30) - 1;
constexpr int64_t kMaxTopk = 1024;
constexpr int kMaxExperts = 2048;
constexpr int64_t kMaxRowK = (int64_t)1 << 20;
constexpr int64_t kMaxRowBytes = (int64_t)1 << 22;
constexpr int64_t kMaxStride = (int64_t)1 << 31;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// ---------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------
constexpr int kSortWaves = 8;                  // x 2048 experts of LDS counters: 64 KB
constexpr int kSortThreads = 64 * kSortWaves;
// Slots up to which one workgroup sorts alone (4096: 7.2 us in one launch and in
// two; 2048: 4.7 and 7; 8192: 11.9 and 7.4).
constexpr int64_t kSortOne = 4096;
constexpr int kSortBlock = 2048;               // slots of a workgroup otherwise, until
constexpr int kSortMaxBlocks = 256;            // there would be more workgroups than this
constexpr int kSortHold = 4;                   // ids a thread loads at a time

// The experts of slots i, i + step, ... (an id outside 0..experts-1: -1), -1
// from `end` on: all loads, then all uses.
template <typename ID>
__device__ inline void load_experts(int (&e)[kSortHold], const ID *ids, int i, int step, int end, int experts)
{
    ID id[kSortHold];
#pragma unroll
    for (int h = 0; h < kSortHold; ++h) id[h] = i + h * step < end ? ids[i + h * step] : (ID)-1;
#pragma unroll
    for (int h = 0; h < kSortHold; ++h) e[h] = id[h] >= 0 && id[h] < (ID)experts ? (int)id[h] : -1;
}

// Lanes of the wave that hold the same expert as this one (all 64 lanes call).
__device__ inline uint64_t same_expert(int e, int bits)
{
    const uint64_t present = __ballot(e >= 0);
    uint64_t m = e >= 0 ? present : ~present;
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((e >> b) & 1);
        m &= (e >> b) & 1 ? set : ~set;
    }
    return m;
}

struct SortArgs {
    const void *ids;
    int32_t *offsets;
    int32_t *slot_row;
    int32_t *counts;      // [blocks][experts], or NULL for one workgroup
    int n;                // slots
    int per_block;        // slots per workgroup, a multiple of kSortThreads
    int experts;
    int bits;             // 2^bits >= experts
};

// Slots per expert of each workgroup's range (integer atomics in LDS: the
// counts do not depend on their order).
template <typename ID>
__global__ void __launch_bounds__(kSortThreads) k_moe_count(SortArgs a)
{
    __shared__ int32_t hist[kMaxExperts];
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads) hist[e] = 0;
    __syncthreads();
    const int beg = blockIdx.x * a.per_block, end = min(beg + a.per_block, a.n);
    for (int i = beg + threadIdx.x; i < end; i += kSortHold * kSortThreads) {
        int e[kSortHold];
        load_experts(e, static_cast<const ID *>(a.ids), i, kSortThreads, end, a.experts);
#pragma unroll
        for (int h = 0; h < kSortHold; ++h)
            if (e[h] >= 0)
                atomicAdd(&hist[e[h]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads)
        a.counts[(int64_t)blockIdx.x * a.experts + e] = hist[e];
}

// Rows of each workgroup's slots.  A wave owns a contiguous part of the
// workgroup's range: it counts that part, the workgroup turns the waves'
// counts and the counts of the workgroups before it into the wave's first row
// of each expert, and the wave walks its part again 64 slots at a time, a
// slot's rank among the 64 being the number of lower lanes with its expert.
// Latency bounds it: the counts of all workgroups are summed by all threads at
// once, kSortHold loads of each in flight (a thread per expert that walked the
// workgroups' counts: 13 us for 65 528 slots and 128 experts, this: 6 us).
template <typename ID>
__global__ void __launch_bounds__(kSortThreads) k_moe_place(SortArgs a)
{
    __shared__ int32_t hist[kSortWaves * kMaxExperts];
    __shared__ int32_t total[kMaxExperts], before[kMaxExperts];
    __shared__ int32_t wave_total[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const ID *ids = static_cast<const ID *>(a.ids);
    const int part = a.per_block / kSortWaves;
    const int beg = min(blockIdx.x * a.per_block + wave * part, a.n), end = min(beg + part, a.n);
    int held[kSortHold];                                    // the part's first 64 kSortHold slots
    load_experts(held, ids, beg + lane, 64, end, a.experts);
    for (int i = tid; i < kSortWaves * a.experts; i += kSortThreads) hist[i] = 0;
    for (int i = tid; i < a.experts; i += kSortThreads) total[i] = before[i] = 0;
    __syncthreads();
    int32_t *mine = hist + wave * a.experts;
    for (int i = beg; i < end; i += 64 * kSortHold) {
        int e[kSortHold];
        if (i == beg)
            for (int h = 0; h < kSortHold; ++h) e[h] = held[h];
        else
            load_experts(e, ids, i + lane, 64, end, a.experts);
#pragma unroll
        for (int h = 0; h < kSortHold; ++h)
            if (e[h] >= 0)
                atomicAdd(&mine[e[h]], 1);
    }
    if (a.counts) {
        const int all = gridDim.x * a.experts, earlier = blockIdx.x * a.experts;
        for (int i = tid; i < all; i += kSortHold * kSortThreads) {
            int c[kSortHold];
#pragma unroll
            for (int h = 0; h < kSortHold; ++h) {
                const int at = i + h * kSortThreads;
                c[h] = at < all ? a.counts[at] : 0;
            }
#pragma unroll
            for (int h = 0; h < kSortHold; ++h) {
                const int at = i + h * kSortThreads;
                if (c[h]) {
                    atomicAdd(&total[at % a.experts], c[h]);
                    if (at < earlier)
                        atomicAdd(&before[at % a.experts], c[h]);
                }
            }
        }
    }
    __syncthreads();

    // exclusive sums over the experts, a thread taking `each` consecutive ones
    const int each = (a.experts + kSortThreads - 1) / kSortThreads;
    const int e0 = min(tid * each, a.experts), e1 = min(e0 + each, a.experts);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        if (!a.counts)
            for (int w = 0; w < kSortWaves; ++w) total[e] += hist[w * a.experts + e];
        sum += total[e];
    }
    const int scan = wave_scan(sum);
    if (lane == 63)
        wave_total[wave] = scan;
    __syncthreads();
    int first = scan - sum;
    for (int w = 0; w < wave; ++w) first += wave_total[w];
    for (int e = e0; e < e1; ++e) {
        if (blockIdx.x == 0) {
            a.offsets[e] = first;
            if (e == a.experts - 1)
                a.offsets[a.experts] = first + total[e];
        }
        int at = first + before[e];
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = hist[w * a.experts + e];
            hist[w * a.experts + e] = at;
            at += c;
        }
        first += total[e];
    }
    __syncthreads();

    for (int i = beg; i < end; i += 64 * kSortHold) {
        int e[kSortHold];
        if (i == beg)
            for (int h = 0; h < kSortHold; ++h) e[h] = held[h];
        else
            load_experts(e, ids, i + lane, 64, end, a.experts);
#pragma unroll
        for (int h = 0; h < kSortHold; ++h) {
            const int slot = i + h * 64 + lane;
            const uint64_t same = same_expert(e[h], a.bits);
            const int lead = __ffsll((unsigned long long)same) - 1;
            int at = 0;
            if (e[h] >= 0 && lane == lead)
                at = atomicAdd(&mine[e[h]], __popcll(same));
            at = __shfl(at, lead);
            if (slot < end)
                a.slot_row[slot] = e[h] >= 0 ? at + __popcll(same & (((uint64_t)1 << lane) - 1)) : -1;
        }
    }
}

int sort_blocks(int64_t n)
{
    return n <= kSortOne ? 1 : (int)min((n + kSortBlock - 1) / kSortBlock, (int64_t)kSortMaxBlocks);
}

qlin_status check_sort(int32_t id_bits, int64_t tokens, int64_t topk, int64_t experts, const void *ids,
                       const int32_t *offsets, const int32_t *slot_row, const void *ws, size_t ws_bytes)
{
    if (id_bits != 32 && id_bits != 64)
        return QLIN_ERR_BAD_ARGUMENT;
    if (tokens < 0 || topk < 1 || topk > kMaxTopk || tokens > kMaxSlots / topk || experts < 1 ||
        experts > kMaxExperts)
        return QLIN_ERR_BAD_SHAPE;
    if (!offsets || (tokens > 0 && (!ids || !slot_row)))
        return QLIN_ERR_NULL_POINTER;
    if (!aligned(ids, id_bits / 8) || !aligned(offsets, 4) || !aligned(slot_row, 4) || !aligned(ws, 4))
        return QLIN_ERR_MISALIGNED;
    const size_t need = qlin_moe_sort_workspace_size(tokens, topk, experts);
    if (need && (!ws || ws_bytes < need))
        return QLIN_ERR_WORKSPACE;
    return QLIN_OK;
}

template <typename ID>
hipError_t launch_sort_id(const SortArgs &a, int blocks, hipStream_t s)
{
    if (a.counts) {
        hipLaunchKernelGGL((k_moe_count<ID>), dim3(blocks), dim3(kSortThreads), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL((k_moe_place<ID>), dim3(blocks), dim3(kSortThreads), 0, s, a);
    return hipGetLastError();
}

SortArgs sort_args(int64_t tokens, int64_t topk, int64_t experts, const void *ids, int32_t *offsets,
                   int32_t *slot_row, void *ws, int blocks)
{
    const int64_t n = tokens * topk;
    int64_t per = (n + blocks - 1) / blocks;
    per = (per + kSortThreads - 1) / kSortThreads * kSortThreads;
    int bits = 0;
    while (((int64_t)1 << bits) < experts) ++bits;
    return SortArgs{ids, offsets, slot_row, blocks > 1 ? static_cast<int32_t *>(ws) : nullptr, (int)n,
                    (int)per, (int)experts, bits};
}

hipError_t launch_sort(int32_t id_bits, int64_t tokens, int64_t topk, int64_t experts, const void *ids,
                       int32_t *offsets, int32_t *slot_row, void *ws, hipStream_t s)
{
    const int blocks = sort_blocks(tokens * topk);
    const SortArgs a = sort_args(tokens, topk, experts, ids, offsets, slot_row, ws, blocks);
    return id_bits == 64 ? launch_sort_id<int64_t>(a, blocks, s) : launch_sort_id<int32_t>(a, blocks, s);
}

// ---------------------------------------------------------------------------
// Rows.  A token belongs to `lanes` consecutive threads (a power of two up
// to the workgroup's 256), each of which takes 16-byte pieces of the row;
// what is left of a row after its 16-byte pieces goes element by element.
// Pieces need only the element's alignment (the hardware loads and stores 16
// bytes at any address), so odd widths and strides take the same path.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;

struct RowArgs {
    const uint8_t *x;       // permute: X; combine: Y; gradient: dOut
    const uint8_t *y;       // gradient: Y
    uint8_t *out;
    const int32_t *slot_row;
    const float *weights;   // combine (NULL: all 1) and its gradient
    const float *scale;     // permute
    float *out_f;           // permute: the rows' scales; gradient: dW
    int64_t ldx, ldy, ldo;  // bytes
    int tokens, topk, rows;
    int cols;               // permute: bytes of a row; otherwise its elements
    int scale_cols;
    int lanes;
};

// Copies a token's row and scales to its slots' rows, as thread `lane` of its
// a.lanes: a row is read once and written topk times.  Bound by those bytes:
// 8191 tokens of 2 KB and 16 scales to 8 rows each 31 us, 4.8 TB/s.
__device__ inline void copy_token(const RowArgs &a, int token, const int32_t *rows, int lane)
{
    const uint8_t *x = a.x + (int64_t)token * a.ldx;
    const int pieces = a.cols >> 4, tail = a.cols & 15;
    for (int p = lane; p < pieces; p += a.lanes) {
        v4i v;
        __builtin_memcpy(&v, x + 16 * (int64_t)p, 16);
        for (int j = 0; j < a.topk; ++j) {
            const int r = rows[j];
            if ((unsigned)r < (unsigned)a.rows)
                __builtin_memcpy(a.out + r * a.ldo + 16 * (int64_t)p, &v, 16);
        }
    }
    for (int i = lane; i < tail; i += a.lanes) {
        const int at = 16 * pieces + i;
        for (int j = 0; j < a.topk; ++j) {
            const int r = rows[j];
            if ((unsigned)r < (unsigned)a.rows)
                a.out[r * a.ldo + at] = x[at];
        }
    }
    for (int c = lane; c < a.scale_cols; c += a.lanes) {
        const float s = a.scale[(int64_t)token * a.scale_cols + c];
        for (int j = 0; j < a.topk; ++j) {
            const int r = rows[j];
            if ((unsigned)r < (unsigned)a.rows)
                a.out_f[(int64_t)r * a.scale_cols + c] = s;
        }
    }
}

__global__ void __launch_bounds__(kRowThreads) k_moe_permute(RowArgs a)
{
    const int token = blockIdx.x * (kRowThreads / a.lanes) + threadIdx.x / a.lanes;
    if (token < a.tokens)
        copy_token(a, token, a.slot_row + (int64_t)token * a.topk, threadIdx.x & (a.lanes - 1));
}

// Sort and copy in one launch, for few slots: each workgroup counts for its
// own slots who comes before them (the ids fit LDS; a wave takes slots, its
// lanes the ids), and then copies its tokens' rows; the last workgroup makes
// the offsets.  Latency bounds it.  Top-8, 128 experts, 2 KB rows, this and the
// two launches: 128 slots 4.7 and 9 us, 1024 7.5 and 9.4, 2048 10.9 and 9.9, but
// 10.8 against 13.0 for a caller who does not replay graphs; beyond, the sort
// counts faster.
constexpr int kFusedSlots = 2048;

template <typename ID>
__global__ void __launch_bounds__(kRowThreads) k_moe_dispatch(SortArgs s, RowArgs a)
{
    __shared__ int32_t expert[kFusedSlots], row[kFusedSlots];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < s.n; i += kSortHold * kRowThreads) {
        int e[kSortHold];
        load_experts(e, static_cast<const ID *>(s.ids), i, kRowThreads, s.n, s.experts);
#pragma unroll
        for (int h = 0; h < kSortHold; ++h)
            if (i + h * kRowThreads < s.n)
                expert[i + h * kRowThreads] = e[h];
    }
    __syncthreads();
    if (blockIdx.x == gridDim.x - 1) {
        // offsets[e]: slots with a smaller expert
        __shared__ int32_t hist[kMaxExperts], total[kRowThreads / 64];
        for (int e = tid; e < s.experts; e += kRowThreads) hist[e] = 0;
        __syncthreads();
        for (int i = tid; i < s.n; i += kRowThreads)
            if (expert[i] >= 0)
                atomicAdd(&hist[expert[i]], 1);
        __syncthreads();
        const int each = (s.experts + kRowThreads - 1) / kRowThreads;
        int sum = 0;
        for (int e = tid * each; e < min((tid + 1) * each, s.experts); ++e) sum += hist[e];
        const int scan = wave_scan(sum);
        if (lane == 63)
            total[wave] = scan;
        __syncthreads();
        int at = scan - sum;
        for (int w = 0; w < wave; ++w) at += total[w];
        for (int e = tid * each; e < min((tid + 1) * each, s.experts); ++e) {
            s.offsets[e] = at;
            at += hist[e];
            if (e == s.experts - 1)
                s.offsets[s.experts] = at;
        }
        return;
    }
    const int per = kRowThreads / a.lanes;                  // tokens of the workgroup
    const int t0 = blockIdx.x * per, first = t0 * a.topk, last = min(first + per * a.topk, s.n);
    // four slots a wave at a time: each id read serves all of them
    for (int i = first + 4 * wave; i < last; i += 4 * kRowThreads / 64) {
        int e[4], before[4] = {};
#pragma unroll
        for (int c = 0; c < 4; ++c) e[c] = expert[min(i + c, last - 1)];
#pragma unroll 4
        for (int j = lane; j < s.n; j += 64) {
            const int f = expert[j];
#pragma unroll
            for (int c = 0; c < 4; ++c) before[c] += f >= 0 && (f < e[c] || (f == e[c] && j < i + c)) ? 1 : 0;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            before[c] = wave_sum(before[c]);
            if (lane == 0 && i + c < last) {
                row[i + c - first] = e[c] >= 0 ? before[c] : -1;
                s.slot_row[i + c] = e[c] >= 0 ? before[c] : -1;
            }
        }
    }
    __syncthreads();
    const int token = t0 + tid / a.lanes;
    if (token < a.tokens)
        copy_token(a, token, row + tid / a.lanes * a.topk, tid & (a.lanes - 1));
}

template <typename T> struct Elem;
template <> struct Elem<float> {
    static __device__ inline float get(float v) { return v; }
    static __device__ inline float put(float v) { return v; }
};
template <> struct Elem<__half> {
    static __device__ inline float get(__half v) { return __half2float(v); }
    static __device__ inline __half put(float v) { return __float2half(v); }
};
template <> struct Elem<uint16_t> {                // bf16 bits
    static __device__ inline float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ inline uint16_t put(float v) { return bf16_bits(v); }
};

// Choices whose rows a thread loads together.
constexpr int kChoices = 4;

// Rows and weights of choices j to j + kChoices of a token; a choice without a
// row has row -1.
__device__ inline void load_choices(int (&row)[kChoices], float (&w)[kChoices], const RowArgs &a, int64_t slot,
                                    int j)
{
#pragma unroll
    for (int c = 0; c < kChoices; ++c) {
        const int r = j + c < a.topk ? a.slot_row[slot + j + c] : -1;
        row[c] = (unsigned)r < (unsigned)a.rows ? r : -1;
        w[c] = a.weights && j + c < a.topk ? a.weights[slot + j + c] : 1.0f;
    }
}

// out[t] = sum_j w[t,j] y[row[t,j]], the choices in order.  Bound by the rows'
// bytes: 8191 tokens of 8 rows of 4 KB 60 us, 4.8 TB/s (a row after another:
// 65 us; 16 tokens 3.8 and 4.2 us, a launch and two latencies).
template <typename T>
__global__ void __launch_bounds__(kRowThreads) k_moe_combine(RowArgs a)
{
    constexpr int V = 16 / sizeof(T);
    const int token = blockIdx.x * (kRowThreads / a.lanes) + threadIdx.x / a.lanes;
    const int lane = threadIdx.x & (a.lanes - 1);
    if (token >= a.tokens)
        return;
    const int64_t slot = (int64_t)token * a.topk;
    uint8_t *out = a.out + (int64_t)token * a.ldo;
    const int pieces = a.cols / V, tail = a.cols % V;
    for (int p = lane; p < pieces; p += a.lanes) {
        float sum[V];
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = 0.0f;
        for (int j = 0; j < a.topk; j += kChoices) {
            int row[kChoices];
            float w[kChoices];
            T v[kChoices][V];
            load_choices(row, w, a, slot, j);
#pragma unroll
            for (int c = 0; c < kChoices; ++c)
                if (row[c] >= 0)
                    __builtin_memcpy(v[c], a.x + row[c] * a.ldx + 16 * (int64_t)p, 16);
#pragma unroll
            for (int c = 0; c < kChoices; ++c)
                if (row[c] >= 0)
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[i] = fmaf(w[c], Elem<T>::get(v[c][i]), sum[i]);
        }
        T o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = Elem<T>::put(sum[i]);
        __builtin_memcpy(out + 16 * (int64_t)p, o, 16);
    }
    for (int i = lane; i < tail; i += a.lanes) {
        const int64_t at = pieces * V + i;
        float sum = 0.0f;
        for (int j = 0; j < a.topk; ++j) {
            const int r = a.slot_row[slot + j];
            if ((unsigned)r < (unsigned)a.rows)
                sum = fmaf(a.weights ? a.weights[slot + j] : 1.0f,
                           Elem<T>::get(reinterpret_cast<const T *>(a.x + r * a.ldx)[at]), sum);
        }
        reinterpret_cast<T *>(out)[at] = Elem<T>::put(sum);
    }
}

// dy[row[t,j]] = w[t,j] dout[t],  dw[t,j] = <dout[t], y[row[t,j]]>: a.lanes
// threads (whole waves) per token, a piece of dout serving kChoices rows, the
// dot products summed over the lanes and then the waves in a fixed order.
// Bound by the bytes of the rows read and written: 8192 tokens of 8 rows of
// 4 KB 104 us, 5.3 TB/s (one wave per token, a row after another: 124 us).
template <typename T>
__global__ void __launch_bounds__(kRowThreads) k_moe_combine_backward(RowArgs a)
{
    constexpr int V = 16 / sizeof(T);
    __shared__ float part[2][kRowThreads / 64][kChoices];
    const int tid = threadIdx.x, lane = tid & (a.lanes - 1);
    const int token = blockIdx.x * (kRowThreads / a.lanes) + tid / a.lanes;
    const bool live = token < a.tokens;
    const uint8_t *dout = a.x + (int64_t)token * a.ldx;
    const int64_t slot = (int64_t)token * a.topk;
    const int pieces = live ? a.cols / V : 0, tail = live ? a.cols % V : 0;
    for (int j = 0, turn = 0; j < a.topk; j += kChoices, turn ^= 1) {
        int row[kChoices] = {-1, -1, -1, -1};
        float w[kChoices], dot[kChoices] = {};
        if (live)
            load_choices(row, w, a, slot, j);
        for (int p = lane; p < pieces; p += a.lanes) {
            T d[V], v[kChoices][V];
            __builtin_memcpy(d, dout + 16 * (int64_t)p, 16);
#pragma unroll
            for (int c = 0; c < kChoices; ++c)
                if (row[c] >= 0)
                    __builtin_memcpy(v[c], a.y + row[c] * a.ldy + 16 * (int64_t)p, 16);
#pragma unroll
            for (int c = 0; c < kChoices; ++c)
                if (row[c] >= 0) {
                    T o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float f = Elem<T>::get(d[i]);
                        dot[c] = fmaf(f, Elem<T>::get(v[c][i]), dot[c]);
                        o[i] = Elem<T>::put(w[c] * f);
                    }
                    __builtin_memcpy(a.out + row[c] * a.ldo + 16 * (int64_t)p, o, 16);
                }
        }
        if (lane < tail) {
            const int at = pieces * V + lane;
            const float f = Elem<T>::get(reinterpret_cast<const T *>(dout)[at]);
#pragma unroll
            for (int c = 0; c < kChoices; ++c)
                if (row[c] >= 0) {
                    dot[c] = fmaf(f, Elem<T>::get(reinterpret_cast<const T *>(a.y + row[c] * a.ldy)[at]), dot[c]);
                    reinterpret_cast<T *>(a.out + row[c] * a.ldo)[at] = Elem<T>::put(w[c] * f);
                }
        }
#pragma unroll
        for (int c = 0; c < kChoices; ++c) dot[c] = wave_sum(dot[c]);
        if ((tid & 63) == 0)
            for (int c = 0; c < kChoices; ++c) part[turn][tid / 64][c] = dot[c];
        __syncthreads();
        // `turn` keeps the next choices' sums apart, so one barrier is enough
        if (live && lane < kChoices && j + lane < a.topk) {
            float sum = 0.0f;
            for (int u = 0; u < a.lanes / 64; ++u) sum += part[turn][tid / 64 + u][lane];
            a.out_f[slot + j + lane] = sum;
        }
    }
}

// Threads per token: enough for one 16-byte piece each, up to a workgroup.
int row_lanes(int64_t bytes)
{
    int l = 16;
    while (l < kRowThreads && 16 * (int64_t)l < bytes) l *= 2;
    return l;
}

dim3 row_grid(const RowArgs &a)
{
    const int per = kRowThreads / a.lanes;
    return dim3((unsigned)((a.tokens + per - 1) / per));
}

// Runs `launch` (grid, arguments) for all tokens, in parts of 2^31 threads at most:
// a grid of 2^32 threads or more is taken modulo that, without an error.
// `advance`: the arguments past so many tokens.
constexpr int kRowBlocks = 1 << 23;

template <typename Launch, typename Advance>
hipError_t launch_rows(RowArgs a, Launch launch, Advance advance)
{
    const int most = (int)std::min<int64_t>((int64_t)kRowBlocks * (kRowThreads / a.lanes), kMaxSlots);
    hipError_t e = hipSuccess;
    for (int left = a.tokens; left > 0 && e == hipSuccess; left -= a.tokens) {
        a.tokens = std::min(left, most);
        launch(row_grid(a), a);
        e = hipGetLastError();
        advance(a, (int64_t)a.tokens);
    }
    return e;
}

qlin_status check_rows(int64_t tokens, int64_t topk, int64_t rows)
{
    if (tokens < 0 || topk < 1 || topk > kMaxTopk || tokens > kMaxSlots / topk || rows < 0 || rows > kMaxSlots)
        return QLIN_ERR_BAD_SHAPE;
    return QLIN_OK;
}

qlin_status check_permute(int64_t row_bytes, const void *X, int64_t ldx, const void *Out, int64_t ldo,
                          const float *scale, int64_t scale_cols, const float *out_scale)
{
    if (row_bytes <= 0 || row_bytes > kMaxRowBytes || scale_cols < 0 || scale_cols > kMaxRowK)
        return QLIN_ERR_BAD_SHAPE;
    if (!X || !Out || (scale_cols > 0 && (!scale || !out_scale)))
        return QLIN_ERR_NULL_POINTER;
    if (ldx < row_bytes || ldo < row_bytes || ldx > kMaxStride || ldo > kMaxStride)
        return QLIN_ERR_BAD_STRIDE;
    if (scale_cols > 0 && (!aligned(scale, 4) || !aligned(out_scale, 4)))
        return QLIN_ERR_MISALIGNED;
    return QLIN_OK;
}

RowArgs permute_args(int64_t tokens, int64_t topk, int64_t rows, int64_t row_bytes, const void *X, int64_t ldx,
                     const int32_t *slot_row, void *Out, int64_t ldo, const float *scale, int64_t scale_cols,
                     float *out_scale)
{
    RowArgs a{};
    a.x = static_cast<const uint8_t *>(X);
    a.out = static_cast<uint8_t *>(Out);
    a.slot_row = slot_row;
    a.scale = scale;
    a.out_f = out_scale;
    a.ldx = ldx;
    a.ldo = ldo;
    a.tokens = (int)tokens;
    a.topk = (int)topk;
    a.rows = (int)rows;
    a.cols = (int)row_bytes;
    a.scale_cols = (int)scale_cols;
    a.lanes = row_lanes(row_bytes);
    return a;
}

hipError_t launch_permute(const RowArgs &a, hipStream_t s)
{
    return launch_rows(
        a, [s](dim3 grid, const RowArgs &p) { hipLaunchKernelGGL(k_moe_permute, grid, dim3(kRowThreads), 0, s, p); },
        [](RowArgs &p, int64_t tokens) {
            p.x += tokens * p.ldx;
            p.slot_row += tokens * p.topk;
            p.scale += p.scale_cols ? tokens * p.scale_cols : 0;
        });
}

// Bytes of an element, 0 for an unknown type.
int elem_size(qlin_row_type rt)
{
    return rt == QLIN_ROW_F32 ? 4 : rt == QLIN_ROW_BF16 || rt == QLIN_ROW_F16 ? 2 : 0;
}

qlin_status combine(qlin_row_type rt, int64_t tokens, int64_t topk, int64_t rows, int64_t K, const void *Y,
                    int64_t ldy, const int32_t *slot_row, const float *weights, void *Out, int64_t ldo,
                    void *stream)
{
    const int es = elem_size(rt);
    if (!es)
        return QLIN_ERR_BAD_ARGUMENT;
    const qlin_status st = check_rows(tokens, topk, rows);
    if (st != QLIN_OK)
        return st;
    if (K <= 0 || K > kMaxRowK)
        return QLIN_ERR_BAD_SHAPE;
    if (tokens == 0)
        return QLIN_OK;
    if ((rows > 0 && !Y) || !slot_row || !Out)
        return QLIN_ERR_NULL_POINTER;
    if (ldy < K || ldo < K || ldy > kMaxStride || ldo > kMaxStride)
        return QLIN_ERR_BAD_STRIDE;
    if (!aligned(Y, es) || !aligned(Out, es) || !aligned(slot_row, 4) || !aligned(weights, 4))
        return QLIN_ERR_MISALIGNED;
    RowArgs a{};
    a.x = static_cast<const uint8_t *>(Y);
    a.out = static_cast<uint8_t *>(Out);
    a.slot_row = slot_row;
    a.weights = weights;
    a.ldx = ldy * es;
    a.ldo = ldo * es;
    a.tokens = (int)tokens;
    a.topk = (int)topk;
    a.rows = (int)rows;
    a.cols = (int)K;
    a.lanes = row_lanes(K * es);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const auto launch = [rt, s](dim3 grid, const RowArgs &p) {
        const dim3 block(kRowThreads);
        switch (rt) {
        case QLIN_ROW_F32: hipLaunchKernelGGL((k_moe_combine<float>), grid, block, 0, s, p); break;
        case QLIN_ROW_BF16: hipLaunchKernelGGL((k_moe_combine<uint16_t>), grid, block, 0, s, p); break;
        case QLIN_ROW_F16: hipLaunchKernelGGL((k_moe_combine<__half>), grid, block, 0, s, p); break;
        }
    };
    const auto advance = [](RowArgs &p, int64_t tokens) {
        p.slot_row += tokens * p.topk;
        p.weights += p.weights ? tokens * p.topk : 0;
        p.out += tokens * p.ldo;
    };
    return launch_rows(a, launch, advance) == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

size_t qlin_moe_sort_workspace_size(int64_t tokens, int64_t topk, int64_t experts)
{
    if (tokens < 0 || topk < 1 || topk > kMaxTopk || tokens > kMaxSlots / topk || experts < 1 ||
        experts > kMaxExperts)
        return 0;
    const int blocks = sort_blocks(tokens * topk);
    return blocks > 1 ? (size_t)blocks * experts * sizeof(int32_t) : 0;
}

qlin_status qlin_moe_sort(int32_t id_bits, int64_t tokens, int64_t topk, int64_t experts,
                          const void *topk_ids, int32_t *group_offsets, int32_t *slot_row,
                          void *workspace, size_t workspace_bytes, void *stream)
{
    const qlin_status st = check_sort(id_bits, tokens, topk, experts, topk_ids, group_offsets, slot_row,
                                      workspace, workspace_bytes);
    if (st != QLIN_OK)
        return st;
    return launch_sort(id_bits, tokens, topk, experts, topk_ids, group_offsets, slot_row, workspace,
                       static_cast<hipStream_t>(stream)) == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
}

qlin_status qlin_moe_permute(int64_t tokens, int64_t topk, int64_t rows, int64_t row_bytes,
                             const void *X, int64_t ldx, const int32_t *slot_row, void *Out,
                             int64_t ldo, const float *scale, int64_t scale_cols, float *out_scale,
                             void *stream)
{
    qlin_status st = check_rows(tokens, topk, rows);
    if (st != QLIN_OK)
        return st;
    if (tokens == 0 || rows == 0)
        return row_bytes <= 0 || row_bytes > kMaxRowBytes ? QLIN_ERR_BAD_SHAPE : QLIN_OK;
    st = check_permute(row_bytes, X, ldx, Out, ldo, scale, scale_cols, out_scale);
    if (st != QLIN_OK)
        return st;
    if (!slot_row)
        return QLIN_ERR_NULL_POINTER;
    if (!aligned(slot_row, 4))
        return QLIN_ERR_MISALIGNED;
    const RowArgs a = permute_args(tokens, topk, rows, row_bytes, X, ldx, slot_row, Out, ldo, scale, scale_cols,
                                   out_scale);
    return launch_permute(a, static_cast<hipStream_t>(stream)) == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
}

qlin_status qlin_moe_dispatch(int32_t id_bits, int64_t tokens, int64_t topk, int64_t experts,
                              const void *topk_ids, int64_t rows, int64_t row_bytes, const void *X,
                              int64_t ldx, void *Out, int64_t ldo, const float *scale,
                              int64_t scale_cols, float *out_scale, int32_t *group_offsets,
                              int32_t *slot_row, void *workspace, size_t workspace_bytes, void *stream)
{
    qlin_status st = check_sort(id_bits, tokens, topk, experts, topk_ids, group_offsets, slot_row, workspace,
                                workspace_bytes);
    if (st != QLIN_OK)
        return st;
    if (rows < tokens * topk || rows > kMaxSlots)
        return QLIN_ERR_BAD_SHAPE;
    if (tokens > 0) {
        st = check_permute(row_bytes, X, ldx, Out, ldo, scale, scale_cols, out_scale);
        if (st != QLIN_OK)
            return st;
    } else if (row_bytes <= 0 || row_bytes > kMaxRowBytes) {
        return QLIN_ERR_BAD_SHAPE;
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    RowArgs a = permute_args(tokens, topk, rows, row_bytes, X, ldx, slot_row, Out, ldo, scale, scale_cols,
                             out_scale);
    if (tokens > 0 && tokens * topk <= kFusedSlots) {
        // at most 16 slots a workgroup (or one token): it counts for all of them
        // (28 tokens, top-7, rows of 128 bytes: 112 slots in one 17.7 us, so 6.1 us)
        while (a.lanes < kRowThreads && kRowThreads / a.lanes * topk > 16) a.lanes *= 2;
        const SortArgs sa = sort_args(tokens, topk, experts, topk_ids, group_offsets, slot_row, nullptr, 1);
        const dim3 grid(row_grid(a).x + 1);
        if (id_bits == 64)
            hipLaunchKernelGGL((k_moe_dispatch<int64_t>), grid, dim3(kRowThreads), 0, s, sa, a);
        else
            hipLaunchKernelGGL((k_moe_dispatch<int32_t>), grid, dim3(kRowThreads), 0, s, sa, a);
        return hipGetLastError() == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
    }
    if (launch_sort(id_bits, tokens, topk, experts, topk_ids, group_offsets, slot_row, workspace, s) !=
        hipSuccess)
        return QLIN_ERR_HIP;
    if (tokens == 0)
        return QLIN_OK;
    return launch_permute(a, s) == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
}

qlin_status qlin_moe_combine(qlin_row_type rt, int64_t tokens, int64_t topk, int64_t rows, int64_t K,
                             const void *Y, int64_t ldy, const int32_t *slot_row, const float *weights,
                             void *Out, int64_t ldo, void *stream)
{
    if (tokens > 0 && !weights)
        return QLIN_ERR_NULL_POINTER;
    return combine(rt, tokens, topk, rows, K, Y, ldy, slot_row, weights, Out, ldo, stream);
}

qlin_status qlin_moe_permute_backward(qlin_row_type rt, int64_t tokens, int64_t topk, int64_t rows,
                                      int64_t K, const void *dOut, int64_t ldo, const int32_t *slot_row,
                                      void *dX, int64_t ldx, void *stream)
{
    return combine(rt, tokens, topk, rows, K, dOut, ldo, slot_row, nullptr, dX, ldx, stream);
}

qlin_status qlin_moe_combine_backward(qlin_row_type rt, int64_t tokens, int64_t topk, int64_t rows,
                                      int64_t K, const void *dOut, int64_t ldo, const void *Y,
                                      int64_t ldy, const int32_t *slot_row, const float *weights,
                                      void *dY, int64_t lddy, float *dW, void *stream)
{
    const int es = elem_size(rt);
    if (!es)
        return QLIN_ERR_BAD_ARGUMENT;
    const qlin_status st = check_rows(tokens, topk, rows);
    if (st != QLIN_OK)
        return st;
    if (K <= 0 || K > kMaxRowK)
        return QLIN_ERR_BAD_SHAPE;
    if (tokens == 0)
        return QLIN_OK;
    if (!dOut || !slot_row || !weights || !dW || (rows > 0 && (!Y || !dY)))
        return QLIN_ERR_NULL_POINTER;
    if (ldo < K || ldy < K || lddy < K || ldo > kMaxStride || ldy > kMaxStride || lddy > kMaxStride)
        return QLIN_ERR_BAD_STRIDE;
    if (!aligned(dOut, es) || !aligned(Y, es) || !aligned(dY, es) || !aligned(slot_row, 4) ||
        !aligned(weights, 4) || !aligned(dW, 4))
        return QLIN_ERR_MISALIGNED;
    RowArgs a{};
    a.x = static_cast<const uint8_t *>(dOut);
    a.y = static_cast<const uint8_t *>(Y);
    a.out = static_cast<uint8_t *>(dY);
    a.out_f = dW;
    a.slot_row = slot_row;
    a.weights = weights;
    a.ldx = ldo * es;
    a.ldy = ldy * es;
    a.ldo = lddy * es;
    a.tokens = (int)tokens;
    a.topk = (int)topk;
    a.rows = (int)rows;
    a.cols = (int)K;
    a.lanes = std::max(row_lanes(K * es), 64);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const auto launch = [rt, s](dim3 grid, const RowArgs &p) {
        const dim3 block(kRowThreads);
        switch (rt) {
        case QLIN_ROW_F32: hipLaunchKernelGGL((k_moe_combine_backward<float>), grid, block, 0, s, p); break;
        case QLIN_ROW_BF16: hipLaunchKernelGGL((k_moe_combine_backward<uint16_t>), grid, block, 0, s, p); break;
        case QLIN_ROW_F16: hipLaunchKernelGGL((k_moe_combine_backward<__half>), grid, block, 0, s, p); break;
        }
    };
    const auto advance = [](RowArgs &p, int64_t tokens) {
        p.x += tokens * p.ldx;
        p.slot_row += tokens * p.topk;
        p.weights += tokens * p.topk;
        p.out_f += tokens * p.topk;
    };
    return launch_rows(a, launch, advance) == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
}

}  // extern "C"
