// Rows of an embedding table by token, with scaling, and the table's gradient.
//
//   out[t] = c s[id_t, g(h)] table[id_t]             (zeros where there is no such row)
//   dtable[v] = c sum_{t : id_t = v} dout[t]
//
// The gradient sorts the positions by token (a stable radix sort, so equal tokens
// stay in order) and sums each token's run in that order: no atomics on values, and
// results do not depend on timing.  A run that crosses the border between two
// workgroups' shares of the sorted positions leaves a partial sum in each; a second
// kernel adds them in four shares, each in order, and the shares in order.  All of it
// moves bytes once; HBM bounds the long calls and the launch the short ones.
#include <algorithm>

#include "qlin_dpp.h"
#include "qlin_elem.h"
#include "qlin_overlap.h"
#include "qlin_sort.h"
#include "qlinear.h"

namespace qlin {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxTokens = ((int64_t)1 << 30) - 1;
constexpr int64_t kMaxVocab = ((int64_t)1 << 22) - 1;       // two digits of 11 bits, and one key for no token
constexpr int64_t kMaxWidth = (int64_t)1 << 20;
constexpr int64_t kMaxStride = (int64_t)1 << 31;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int elem_size(qlin_row_type rt)
{
    return rt == QLIN_ROW_F32 ? 4 : rt == QLIN_ROW_BF16 || rt == QLIN_ROW_F16 ? 2 : 0;
}

// Token `t`'s row, -1 for none.
__device__ inline int row_of(const void *ids, int id_bits, int64_t t, int vocab)
{
    const int64_t id = id_bits == 64 ? static_cast<const int64_t *>(ids)[t] : static_cast<const int32_t *>(ids)[t];
    return id >= 0 && id < vocab ? (int)id : -1;
}

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------
struct LookArgs {
    const void *ids;
    const uint8_t *table;
    const float *scale;        // [vocab][scale_cols], or NULL
    uint8_t *out;
    int64_t ldt, ldo;          // bytes
    int64_t tokens;
    float factor;
    int vocab, width, scale_cols, id_bits, lanes;
};

// Table elements as fp32: plain ones, int8 and e4m3 codes.
template <typename T> struct Code : Elem<T> {};
template <> struct Code<int8_t> {
    static __device__ inline float get(int8_t v) { return (float)v; }
};
template <> struct Code<uint8_t> {             // e4m3
    static __device__ inline float get(uint8_t v) { return __builtin_amdgcn_cvt_f32_fp8((int)v, 0); }
};

// A token belongs to `lanes` consecutive threads, each of which takes pieces of 16 bytes of the output.  Bytes bound it:
// 8192 rows of 5120 in bf16 28.9 us, 5.8 TB/s; 16 rows 3.8 us, which is a launch.
template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) k_embedding(LookArgs a)
{
    constexpr int E = 16 / sizeof(O);
    const int64_t token = (int64_t)blockIdx.x * (kThreads / a.lanes) + threadIdx.x / a.lanes;
    const int lane = threadIdx.x & (a.lanes - 1);
    if (token >= a.tokens)
        return;
    const int row = row_of(a.ids, a.id_bits, token, a.vocab);
    const T *x = reinterpret_cast<const T *>(a.table + (row < 0 ? 0 : row) * a.ldt);
    O *out = reinterpret_cast<O *>(a.out + token * a.ldo);
    const float *scale = a.scale ? a.scale + (int64_t)(row < 0 ? 0 : row) * a.scale_cols : nullptr;
    for (int at = lane * E; at < a.width; at += a.lanes * E) {
        const int n = min(E, a.width - at);
        float v[E] = {};
        if (row >= 0) {
            T t[E] = {};
            if (n == E)
                __builtin_memcpy(t, x + at, sizeof(t));
            else
#pragma unroll
                for (int i = 0; i < E; ++i)
                    if (i < n)
                        t[i] = x[at + i];
            // (a piece of 8 lies within one group of 128)
            const float s = !scale ? 1.0f : scale[a.scale_cols == 1 ? 0 : at >> 7];
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = Code<T>::get(t[i]) * s * a.factor;
        }
        if (n == E) {
            const v4i o = value_piece<O>(v);
            __builtin_memcpy(out + at, &o, 16);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (i < n)
                    out[at + i] = Elem<O>::put(v[i]);
        }
    }
}

// ---------------------------------------------------------------------------
// Sort of positions by token: least significant digit first, a counting sort a digit.  As pairs (key, position);
// the key of a position without a row is the vocabulary's size, which comes last.  Its launches are short and
// leave most of the GPU idle: the table's zeros are written beside them, a share in each (a table of 131072 rows of 2048
// in bf16, 537 MB: 100 us for both, 78 for the zeros alone).
// ---------------------------------------------------------------------------
constexpr int kDigitBits = 11;
constexpr int kSortOne = 4096;                 // positions up to which one workgroup sorts alone

// Zeros in rows `from` .. `to` - 1 of `width` elements, the last of all (`rows` - 1) of `last`; in workgroups behind
// the `skip` that have other work.
struct FillArgs {
    uint8_t *out;
    int64_t ldo, rows, from, to;               // ldo in bytes
    int width, last, size, skip;               // size: bytes of an element
};

__device__ inline void fill(const FillArgs &f)
{
    for (int64_t row = f.from + blockIdx.x - f.skip; row < f.to; row += gridDim.x - f.skip) {
        uint8_t *o = f.out + row * f.ldo;
        const int64_t end = (int64_t)(row == f.rows - 1 ? f.last : f.width) * f.size;
        for (int64_t at = threadIdx.x * 16; at < end; at += blockDim.x * 16) {
            if (at + 16 <= end) {
                const v4i z{0, 0, 0, 0};
                __builtin_memcpy(o + at, &z, 16);
            } else {
                for (int64_t j = at; j < end; j += 2) *reinterpret_cast<uint16_t *>(o + j) = 0;
            }
        }
    }
}

__global__ void __launch_bounds__(kSortThreads) k_fill(FillArgs f) { fill(f); }

struct SortArgs {
    const void *ids;           // the first digit's input, or NULL
    const int2 *in;            // the later ones'
    int2 *out;
    int32_t *counts;           // [blocks][digits], or NULL for one workgroup
    int n, per_block, blocks, vocab, id_bits;
    int shift, digits;         // digit = (key >> shift) % digits, a power of two
};

__device__ inline SortRange range_of(const SortArgs &a) { return SortRange{a.n, a.per_block, a.blocks, a.counts}; }

__device__ inline int2 pair_at(const SortArgs &a, int i)
{
    if (!a.ids)
        return a.in[i];
    const int r = row_of(a.ids, a.id_bits, i, a.vocab);
    return make_int2(r < 0 ? a.vocab : r, i);
}

// Positions per digit of each workgroup's range (integer atomics: their order does not matter).
__global__ void __launch_bounds__(kSortThreads) k_sort_count(SortArgs a, FillArgs f)
{
    extern __shared__ int32_t hist[];
    if ((int)blockIdx.x >= a.blocks) {
        fill(f);
        return;
    }
    count(range_of(a), a.shift, a.digits, hist, [&](int i) { return pair_at(a, i).x; });
}

__global__ void __launch_bounds__(kSortThreads) k_sort_place(SortArgs a, FillArgs f)
{
    extern __shared__ int32_t hist[];
    if ((int)blockIdx.x >= a.blocks) {
        fill(f);
        return;
    }
    place(range_of(a), a.shift, a.digits, hist, [&](int i) { return pair_at(a, i); }, [&](int at, int2 p) { a.out[at] = p; });
}

// Few positions: both digits (of `low` bits, and the others) in one launch, the pairs in LDS between them.
__global__ void __launch_bounds__(kSortThreads) k_sort_one(SortArgs a, int high, FillArgs f)
{
    extern __shared__ int32_t hist[];
    __shared__ int2 pairs[kSortOne];
    if (blockIdx.x > 0) {
        fill(f);
        return;
    }
    if (high == 1) {
        place(range_of(a), 0, a.digits, hist, [&](int i) { return pair_at(a, i); }, [&](int at, int2 p) { a.out[at] = p; });
        return;
    }
    place(range_of(a), 0, a.digits, hist, [&](int i) { return pair_at(a, i); }, [&](int at, int2 p) { pairs[at] = p; });
    __syncthreads();
    place(range_of(a), a.shift, high, hist, [&](int i) { return pairs[i]; }, [&](int at, int2 p) { a.out[at] = p; });
}

// ---------------------------------------------------------------------------
// Sums of the sorted positions' rows
// ---------------------------------------------------------------------------
constexpr int kChunk = 16;     // sorted positions of a workgroup
constexpr int kAtOnce = 8;     // of them whose rows are on their way together

struct SumArgs {
    const int2 *pairs;         // sorted
    const uint8_t *dout;
    uint8_t *out;
    float *part;               // [chunks][2][width]: the run that came in, the run that goes on
    int64_t ldd, ldo;          // bytes
    float factor;
    int n, vocab, width, add;
};

// The n first of E elements as fp32, the others 0.
template <typename T, int E>
__device__ inline void load_values(float (&v)[E], const T *p, int n)
{
    T t[E];
    if (n == E) {
        __builtin_memcpy(t, p, sizeof(t));
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) t[i] = i < n ? p[i] : Elem<T>::put(0.0f);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = Elem<T>::get(t[i]);
}

template <typename T, int E>
__device__ inline void store_values(T *p, const float (&v)[E], int n)
{
    T t[E];
#pragma unroll
    for (int i = 0; i < E; ++i) t[i] = Elem<T>::put(v[i]);
    if (n == E)
        __builtin_memcpy(p, t, sizeof(t));
    else
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < n)
                p[i] = t[i];
}

// A token's sum to its row of the table (added to what it holds where the caller wants that).
template <typename O, int E>
__device__ inline void store_row(const SumArgs &a, int row, int at, int n, const float (&sum)[E])
{
    O *o = reinterpret_cast<O *>(a.out + row * a.ldo) + at;
    float v[E] = {};
    if (a.add)
        load_values<O, E>(v, o, n);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = a.add ? fmaf(sum[i], a.factor, v[i]) : sum[i] * a.factor;
    store_values<O, E>(o, v, n);
}

// kChunk sorted positions and 16 bytes of a row for each thread a workgroup.  The rows are read in no order and bound it:
// 16384 of 2048 in bf16, 67 MB, 37 us (16 of them at once took as long).
template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) k_sum(SumArgs a)
{
    constexpr int E = 16 / sizeof(T);
    __shared__ int2 pair[kChunk + 2];          // with the neighbours on both sides
    const int first = blockIdx.x * kChunk, count = min(kChunk, a.n - first);
    if (threadIdx.x < kChunk + 2) {
        const int i = first + (int)threadIdx.x - 1;
        pair[threadIdx.x] = i >= 0 && i < a.n ? a.pairs[i] : make_int2(-1, 0);
    }
    __syncthreads();
    const int at = (blockIdx.y * kThreads + threadIdx.x) * E, n = min(E, a.width - at);
    if (n <= 0)
        return;
    float sum[E] = {};
    int began = 0;                             // where the run began
#pragma unroll 1
    for (int j = 0; j < count; j += kAtOnce) {
        v4i t[kAtOnce];                        // (as they come: values taken out here would wait for each load)
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            t[u] = v4i{0, 0, 0, 0};
            if (j + u < count && pair[j + u + 1].x < a.vocab) {
                const T *p = reinterpret_cast<const T *>(a.dout + pair[j + u + 1].y * a.ldd) + at;
                if (n == E) {
                    t[u] = load_piece(p);
                } else {
                    T e[E];
#pragma unroll
                    for (int i = 0; i < E; ++i) e[i] = i < n ? p[i] : Elem<T>::put(0.0f);
                    __builtin_memcpy(&t[u], e, 16);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int p = j + u + 1, key = j + u < count ? pair[p].x : a.vocab;
            if (key >= a.vocab)
                continue;
            float v[E];
            piece_values<T>(v, t[u]);
#pragma unroll
            for (int i = 0; i < E; ++i) sum[i] += v[i];
            const bool ends = pair[p + 1].x != key;
            if (!ends && j + u + 1 < count)
                continue;
            const bool came = began == 0 && pair[0].x == key;
            if (ends && !came)
                store_row<O, E>(a, key, at, n, sum);
            else
                store_values<float, E>(a.part + ((int64_t)blockIdx.x * 2 + (came ? 0 : 1)) * a.width + at, sum, n);
            began = j + u + 1;
#pragma unroll
            for (int i = 0; i < E; ++i) sum[i] = 0.0f;
        }
    }
}

// The runs that cross chunks: the workgroup of the chunk where one begins adds its parts, each wave a share of them in
// order (a token of 950 positions has 60), then the waves' sums in order.
constexpr int kJoinWaves = 4, kJoinWidth = 256;

template <typename O>
__global__ void __launch_bounds__(64 * kJoinWaves) k_join(SumArgs a)
{
    __shared__ float sums[kJoinWaves][kJoinWidth];
    const int last = (blockIdx.x + 1) * kChunk - 1;         // the chunk's last position
    if (last + 1 >= a.n)
        return;
    const int key = a.pairs[last].x, next = a.pairs[last + 1].x, before = blockIdx.x ? a.pairs[last - kChunk].x : -1;
    if (key >= a.vocab || next != key || before == key)
        return;                                             // (a run that fills the chunk began in an earlier one)
    // the chunks that begin with the token, counted 64 at a time
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int parts = 0;
    for (int more = 64; more == 64; parts += more) {
        const int64_t i = last + 1 + (int64_t)(parts + lane) * kChunk;
        more = __popcll(__ballot(i < a.n && a.pairs[i].x == key));
    }
    const int at = blockIdx.y * kJoinWidth + lane * 4, n = min(4, a.width - at);
    // part 0 is the run's beginning in this chunk, part p its piece in the p-th chunk behind
    const int share = (parts + kJoinWaves) / kJoinWaves, end = min((wave + 1) * share, parts + 1);
    float sum[4] = {};
    if (n > 0)
        for (int j = wave * share; j < end; j += 8) {
            float v[8][4];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (j + u < end)
                    load_values<float, 4>(v[u], a.part + ((int64_t)(blockIdx.x + j + u) * 2 + (j + u == 0 ? 1 : 0)) * a.width + at, n);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (j + u < end)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[i] += v[u][i];
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[wave][4 * lane + i] = sum[i];
    __syncthreads();
    if (wave > 0 || n <= 0)
        return;
    for (int w = 1; w < kJoinWaves; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += sums[w][4 * lane + i];
    store_row<O, 4>(a, key, at, n, sum);
}

int sort_blocks(int64_t n) { return n <= kSortOne ? 1 : sort_parts(n); }

int64_t chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }
int64_t column_blocks(int64_t width) { return (width + 255) / 256; }           // of the join, the most

// A launch has fewer than 2^32 threads.
bool sums_fit(int64_t n, int64_t width) { return chunks(n) * column_blocks(width) < (int64_t)1 << 24; }

bool backward_shape(int64_t n, int64_t vocab, int64_t width)
{
    return n >= 0 && n <= kMaxTokens / 4 && vocab > 0 && vocab <= kMaxVocab && width > 0 && width <= kMaxWidth &&
           sums_fit(n, width);
}

// Digits of the sort: passes of `low` bits and the others.
struct Digits {
    int passes, low, bits;
};

Digits digits_of(int64_t vocab)
{
    Digits d{1, 0, 0};
    while (((int64_t)1 << d.bits) <= vocab) ++d.bits;       // keys 0 .. vocab
    d.passes = d.bits > kDigitBits ? 2 : 1;
    d.low = (d.bits + d.passes - 1) / d.passes;
    return d;
}

// Two buffers of pairs, the counts and the partial sums.
struct Space {
    size_t pairs, counts, part, bytes;
};

Space space(int64_t n, int64_t vocab, int64_t width)
{
    Space s;
    s.pairs = ((size_t)n * sizeof(int2) + 15) / 16 * 16;
    s.counts = sort_blocks(n) > 1 ? ((size_t)sort_blocks(n) << digits_of(vocab).low) * sizeof(int32_t) : 0;
    s.counts = (s.counts + 15) / 16 * 16;
    s.part = (size_t)chunks(n) * 2 * width * sizeof(float);
    s.bytes = 2 * s.pairs + s.counts + s.part;
    return s;
}

// Workgroups that write zeros beside `blocks` others, and their share of the rows.
constexpr int kFillBlocks = 2048;

FillArgs share_of(FillArgs f, int part, int parts, int blocks)
{
    f.from = f.rows * part / parts;
    f.to = f.rows * (part + 1) / parts;
    f.skip = blocks;
    return f;
}

int fill_blocks(const FillArgs &f) { return (int)std::min<int64_t>(f.to - f.from, kFillBlocks); }

// The sorted pairs lie in the returned buffer, a or b.  `f` is filled by the launches together (no rows: none).
hipError_t launch_sort(const void *ids, int32_t id_bits, int64_t n, int64_t vocab, int2 *a, int2 *b, int32_t *counts,
                       const FillArgs &f, hipStream_t s, int2 **sorted)
{
    const Digits d = digits_of(vocab);
    const int blocks = sort_blocks(n);
    const int per = sort_share(n, blocks);
    SortArgs sa{ids, nullptr, a, blocks > 1 ? counts : nullptr, (int)n, per, blocks, (int)vocab, id_bits, 0, 1 << d.low};
    *sorted = a;
    if (blocks == 1) {
        const FillArgs g = share_of(f, 0, 1, 1);
        sa.shift = d.low;
        hipLaunchKernelGGL(k_sort_one, dim3(1 + fill_blocks(g)), dim3(kSortThreads), place_lds(1 << d.low), s, sa,
                           1 << (d.bits - d.low), g);
        return hipGetLastError();
    }
    for (int p = 0; p < d.passes; ++p) {
        FillArgs g = share_of(f, 2 * p, 2 * d.passes, blocks);
        hipLaunchKernelGGL(k_sort_count, dim3(blocks + fill_blocks(g)), dim3(kSortThreads), sa.digits * sizeof(int32_t), s,
                           sa, g);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        g = share_of(f, 2 * p + 1, 2 * d.passes, blocks);
        hipLaunchKernelGGL(k_sort_place, dim3(blocks + fill_blocks(g)), dim3(kSortThreads), place_lds(sa.digits), s, sa, g);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        *sorted = sa.out;
        sa.ids = nullptr;
        sa.in = sa.out;
        sa.out = b;
        sa.shift = d.low;
        sa.digits = 1 << (d.bits - d.low);
    }
    return hipSuccess;
}

template <typename T, typename O>
hipError_t launch_sums(const SumArgs &a, hipStream_t s)
{
    constexpr int kCols = 16 / sizeof(T) * kThreads;
    const dim3 grid((unsigned)chunks(a.n), (unsigned)((a.width + kCols - 1) / kCols));
    hipLaunchKernelGGL((k_sum<T, O>), grid, dim3(kThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || grid.x == 1)
        return e;
    hipLaunchKernelGGL((k_join<O>), dim3(grid.x - 1, (unsigned)((a.width + kJoinWidth - 1) / kJoinWidth)),
                       dim3(64 * kJoinWaves), 0, s, a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_look(qlin_row_type ot, const LookArgs &a, dim3 grid, hipStream_t s)
{
    switch (ot) {
    case QLIN_ROW_F32: hipLaunchKernelGGL((k_embedding<T, float>), grid, dim3(kThreads), 0, s, a); break;
    case QLIN_ROW_BF16: hipLaunchKernelGGL((k_embedding<T, uint16_t>), grid, dim3(kThreads), 0, s, a); break;
    case QLIN_ROW_F16: hipLaunchKernelGGL((k_embedding<T, __half>), grid, dim3(kThreads), 0, s, a); break;
    }
    return hipGetLastError();
}

int table_size(qlin_table_type tt)
{
    switch (tt) {
    case QLIN_TABLE_F32: return 4;
    case QLIN_TABLE_BF16:
    case QLIN_TABLE_F16: return 2;
    case QLIN_TABLE_INT8:
    case QLIN_TABLE_E4M3: return 1;
    }
    return 0;
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

qlin_status qlin_embedding(qlin_table_type tt, qlin_row_type ot, int32_t id_bits, int64_t tokens, int64_t vocab,
                           int64_t width, const void *ids, const void *table, int64_t ldt, const float *row_scale,
                           int64_t scale_cols, float scale, void *Out, int64_t ldo, void *stream)
{
    const int ts = table_size(tt), os = elem_size(ot);
    if (!ts || !os || (id_bits != 32 && id_bits != 64))
        return QLIN_ERR_BAD_ARGUMENT;
    if (tokens < 0 || tokens > kMaxTokens || vocab <= 0 || vocab >= ((int64_t)1 << 31) || width <= 0 ||
        width > kMaxWidth || (scale_cols != 0 && scale_cols != 1 && scale_cols * 128 != width))
        return QLIN_ERR_BAD_SHAPE;
    if (tokens == 0)
        return QLIN_OK;
    if (!ids || !table || !Out || (scale_cols > 0 && !row_scale))
        return QLIN_ERR_NULL_POINTER;
    if (ldt < width || ldo < width || ldt > kMaxStride || ldo > kMaxStride)
        return QLIN_ERR_BAD_STRIDE;
    if (!aligned(ids, id_bits / 8) || !aligned(table, ts) || !aligned(Out, os) || !aligned(row_scale, 4))
        return QLIN_ERR_MISALIGNED;
    if (overlaps({Region{Out, tokens, width * os, ldo * os}},
                 {Region{table, vocab, width * ts, ldt * ts}, flat(ids, tokens * (id_bits / 8)),
                  flat(row_scale, 4 * vocab * scale_cols)}))
        return QLIN_ERR_BAD_ARGUMENT;
    LookArgs a{};
    a.ids = ids;
    a.table = static_cast<const uint8_t *>(table);
    a.scale = scale_cols ? row_scale : nullptr;
    a.out = static_cast<uint8_t *>(Out);
    a.ldt = ldt * ts;
    a.ldo = ldo * os;
    a.factor = scale;
    a.vocab = (int)vocab;
    a.width = (int)width;
    a.scale_cols = (int)scale_cols;
    a.id_bits = id_bits;
    a.lanes = 16;
    while (a.lanes < kThreads && (int64_t)a.lanes * 16 < width * os) a.lanes *= 2;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t per = kThreads / a.lanes, most = ((int64_t)1 << 23) * per;      // 2^31 threads a launch
    hipError_t e = hipSuccess;
    for (int64_t left = tokens; left > 0 && e == hipSuccess; left -= a.tokens) {
        a.tokens = std::min(left, most);
        const dim3 grid((unsigned)((a.tokens + per - 1) / per));
        switch (tt) {
        case QLIN_TABLE_F32: e = launch_look<float>(ot, a, grid, s); break;
        case QLIN_TABLE_BF16: e = launch_look<uint16_t>(ot, a, grid, s); break;
        case QLIN_TABLE_F16: e = launch_look<__half>(ot, a, grid, s); break;
        case QLIN_TABLE_INT8: e = launch_look<int8_t>(ot, a, grid, s); break;
        case QLIN_TABLE_E4M3: e = launch_look<uint8_t>(ot, a, grid, s); break;
        }
        a.ids = static_cast<const uint8_t *>(a.ids) + a.tokens * (id_bits / 8);
        a.out += a.tokens * a.ldo;
    }
    return e == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
}

size_t qlin_embedding_backward_workspace_size(int64_t tokens, int64_t vocab, int64_t width)
{
    return tokens > 0 && backward_shape(tokens, vocab, width) ? space(tokens, vocab, width).bytes : 0;
}

qlin_status qlin_embedding_backward(qlin_row_type rt, qlin_row_type ot, int32_t id_bits, int64_t tokens,
                                    int64_t vocab, int64_t width, const void *ids, const void *dOut, int64_t ldd,
                                    float scale, int32_t accumulate, void *dTable, int64_t ldt, void *workspace,
                                    size_t workspace_bytes, void *stream)
{
    const int es = elem_size(rt), os = elem_size(ot);
    if (!es || !os || (ot != rt && ot != QLIN_ROW_F32) || (id_bits != 32 && id_bits != 64))
        return QLIN_ERR_BAD_ARGUMENT;
    if (!backward_shape(tokens, vocab, width))
        return QLIN_ERR_BAD_SHAPE;
    if (!dTable || (tokens > 0 && (!ids || !dOut)))
        return QLIN_ERR_NULL_POINTER;
    if (ldt < width || ldt > kMaxStride || (tokens > 0 && (ldd < width || ldd > kMaxStride)))
        return QLIN_ERR_BAD_STRIDE;
    if (!aligned(dTable, os) || !aligned(ids, id_bits / 8) || !aligned(dOut, es) || !aligned(workspace, 16))
        return QLIN_ERR_MISALIGNED;
    const size_t need = qlin_embedding_backward_workspace_size(tokens, vocab, width);
    if (need && (!workspace || workspace_bytes < need))
        return QLIN_ERR_WORKSPACE;
    if (overlaps({Region{dTable, vocab, width * os, ldt * os}, flat(workspace, need)},
                 {Region{dOut, tokens, width * es, ldd * es}, flat(ids, tokens * (id_bits / 8))}))
        return QLIN_ERR_BAD_ARGUMENT;
    hipStream_t s = static_cast<hipStream_t>(stream);
    FillArgs f{};
    if (!accumulate) {
        // (rows without gaps are as rows of 16384)
        const bool whole = ldt == width;
        const int64_t all = vocab * width, row = whole ? 16384 : width;
        f.out = static_cast<uint8_t *>(dTable);
        f.ldo = (whole ? row : ldt) * os;
        f.rows = (all + row - 1) / row;
        f.width = (int)row;
        f.last = (int)(all - (f.rows - 1) * row);
        f.size = os;
    }
    if (tokens == 0) {
        if (accumulate)
            return QLIN_OK;
        const FillArgs g = share_of(f, 0, 1, 0);
        hipLaunchKernelGGL(k_fill, dim3(fill_blocks(g)), dim3(kSortThreads), 0, s, g);
        return hipGetLastError() == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
    }
    const Space sp = space(tokens, vocab, width);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    SumArgs a{};
    int2 *sorted = nullptr;
    if (launch_sort(ids, id_bits, tokens, vocab, reinterpret_cast<int2 *>(ws), reinterpret_cast<int2 *>(ws + sp.pairs),
                    reinterpret_cast<int32_t *>(ws + 2 * sp.pairs), f, s, &sorted) != hipSuccess)
        return QLIN_ERR_HIP;
    a.pairs = sorted;
    a.dout = static_cast<const uint8_t *>(dOut);
    a.out = static_cast<uint8_t *>(dTable);
    a.part = reinterpret_cast<float *>(ws + 2 * sp.pairs + sp.counts);
    a.ldd = ldd * es;
    a.ldo = ldt * os;
    a.factor = scale;
    a.n = (int)tokens;
    a.vocab = (int)vocab;
    a.width = (int)width;
    a.add = accumulate != 0;
    hipError_t e;
    if (ot == QLIN_ROW_F32)
        e = rt == QLIN_ROW_F32 ? launch_sums<float, float>(a, s)
            : rt == QLIN_ROW_BF16 ? launch_sums<uint16_t, float>(a, s)
                                  : launch_sums<__half, float>(a, s);
    else
        e = rt == QLIN_ROW_BF16 ? launch_sums<uint16_t, uint16_t>(a, s) : launch_sums<__half, __half>(a, s);
    return e == hipSuccess ? QLIN_OK : QLIN_ERR_HIP;
}

}  // extern "C"
