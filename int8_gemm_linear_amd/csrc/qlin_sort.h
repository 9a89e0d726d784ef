// One digit of a stable counting sort over several workgroups: each counts its range, and each then places its pairs
// behind those of the workgroups, waves and lanes before it.  No order of atomics reaches a result.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "qlin_moe_scan.h"

namespace qlin {

constexpr int kSortWaves = 8, kSortThreads = 64 * kSortWaves;
constexpr int kSortBlock = 2048;               // elements of a workgroup, until
constexpr int kSortMaxBlocks = 256;            // there would be more workgroups than this

inline int sort_parts(int64_t n) { return (int)std::min<int64_t>((n + kSortBlock - 1) / kSortBlock, kSortMaxBlocks); }

// Elements of each of `blocks` workgroups.
inline int sort_share(int64_t n, int blocks)
{
    const int64_t per = (n + blocks - 1) / blocks;
    return (int)((per + kSortThreads - 1) / kSortThreads * kSortThreads);
}

struct SortRange {
    int n, per_block, blocks;
    int32_t *counts;           // [blocks][digits], or NULL for one workgroup
};

// Elements per digit of the workgroup's range; key(i) is element i's, hist [digits] in LDS.
template <typename Key>
__device__ inline void count(const SortRange &a, int shift, int digits, int32_t *hist, Key key)
{
    for (int d = threadIdx.x; d < digits; d += kSortThreads) hist[d] = 0;
    __syncthreads();
    const int beg = (int)min((int64_t)blockIdx.x * a.per_block, (int64_t)a.n), end = min(beg + a.per_block, a.n);
#pragma unroll 4
    for (int i = beg + threadIdx.x; i < end; i += kSortThreads) atomicAdd(&hist[(key(i) >> shift) & (digits - 1)], 1);
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kSortThreads) a.counts[(int64_t)blockIdx.x * digits + d] = hist[d];
}

// LDS of `digits`: [waves][digits], twice [digits].
constexpr size_t place_lds(int digits) { return (size_t)(kSortWaves + 2) * digits * sizeof(int32_t); }

// One digit: get(i) is pair i (its key in x), put(place, pair) takes it.  Behind the waves' counts `hist` ends with the
// digits' totals over all workgroups.  A wave owns a contiguous part of the workgroup's range; a
// pair's place is the first place of its digit for the wave, plus those of the wave before it, 64 at a time, plus the
// lower lanes with its digit.
template <typename Get, typename Put>
__device__ inline void place(const SortRange &a, int shift, int digits, int32_t *hist, Get get, Put put)
{
    __shared__ int32_t wave_total[kSortWaves];
    int32_t *total = hist + kSortWaves * digits, *before = total + digits;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, mask = digits - 1;
    const int part = a.per_block / kSortWaves;
    const int beg = (int)min((int64_t)blockIdx.x * a.per_block + wave * part, (int64_t)a.n), end = min(beg + part, a.n);
    for (int i = tid; i < (kSortWaves + 2) * digits; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    int32_t *mine = hist + wave * digits;
#pragma unroll 4
    for (int i = beg + lane; i < end; i += 64) atomicAdd(&mine[(get(i).x >> shift) & mask], 1);
    if (a.counts) {
        const int all = a.blocks * digits, earlier = blockIdx.x * digits;
#pragma unroll 4
        for (int i = tid; i < all; i += kSortThreads) {
            const int c = a.counts[i];
            if (c) {
                atomicAdd(&total[i & mask], c);
                if (i < earlier)
                    atomicAdd(&before[i & mask], c);
            }
        }
    }
    __syncthreads();
    const int each = (digits + kSortThreads - 1) / kSortThreads;
    const int d0 = min(tid * each, digits), d1 = min(d0 + each, digits);
    int sum = 0;
    for (int d = d0; d < d1; ++d) {
        if (!a.counts)
            for (int w = 0; w < kSortWaves; ++w) total[d] += hist[w * digits + d];
        sum += total[d];
    }
    const int scan = wave_scan(sum);
    if (lane == 63)
        wave_total[wave] = scan;
    __syncthreads();
    int first = scan - sum;
    for (int w = 0; w < wave; ++w) first += wave_total[w];
    for (int d = d0; d < d1; ++d) {
        int at = first + before[d];
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = hist[w * digits + d];
            hist[w * digits + d] = at;
            at += c;
        }
        first += total[d];
    }
    __syncthreads();
    const int bits = __ffs(digits) - 1;
    for (int i = beg; i < end; i += 64) {
        const bool there = i + lane < end;
        const int2 p = there ? get(i + lane) : make_int2(0, 0);
        const int d = (p.x >> shift) & mask;
        uint64_t same = __ballot(there);
        same = there ? same : ~same;
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((d >> b) & 1);
            same &= (d >> b) & 1 ? set : ~set;
        }
        const int lead = __ffsll((unsigned long long)same) - 1;
        int at = 0;
        if (there && lane == lead)
            at = atomicAdd(&mine[d], __popcll(same));
        at = __shfl(at, lead);
        if (there)
            put(at + __popcll(same & (((uint64_t)1 << lane) - 1)), p);
    }
}

}  // namespace qlin
