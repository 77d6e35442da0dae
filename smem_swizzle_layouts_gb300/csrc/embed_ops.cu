// Rows of a token table times a factor, and the table's gradient: the product
// of a one-hot operand with the table, and its transpose with the rows'
// gradient. Contracts are in include/gemm_gb300.h.
//
//   D_t = a table[id_t],   dtable_v (+)= a sum of dD_t over the t with id_t = v
//
// The gradient sorts the tokens by id (a stable counting sort by digits of the
// id), cuts the sorted list into chunks, sums runs of one id within a chunk and
// joins those that pass a chunk's end: every sum has a fixed order, no atomic
// adds a floating-point number, and a frequent token's thousands of rows are
// spread over as many blocks as any others. Sums are fp32, rounded once.
// Bound by memory and, in the sort, by latency: 16384 rows of 2048 bf16 into a
// table of 32768 in 53 us, 30 by the bytes of the rows and the table (36 of all
// traffic, with the parts of runs that are cut).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/gemm_gb300.h"
#include "elements.cuh"
#include "host.h"

using namespace g300;

namespace {

// ---------------------------------------------------------------- rows

constexpr int kEmbedThreads = 256;
constexpr int kEmbedItems = 4;  // items a thread has in flight

// VEC neighbouring elements by accesses of up to 16 bytes.
template <typename T, int VEC>
union Vector {
    static constexpr int BYTES = VEC * static_cast<int>(sizeof(T));
    T e[VEC];
    uint4 w16[BYTES >= 16 ? BYTES / 16 : 1];
    uint2 w8;
    __device__ __forceinline__ Vector() {}
    __device__ __forceinline__ void load(const T *p)
    {
        if constexpr (BYTES >= 16) {
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i)
                w16[i] = reinterpret_cast<const uint4 *>(p)[i];
        } else if constexpr (BYTES == 8) {
            w8 = *reinterpret_cast<const uint2 *>(p);
        } else {
            e[0] = *p;
        }
    }
    __device__ __forceinline__ void store(T *p) const
    {
        if constexpr (BYTES >= 16) {
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i)
                reinterpret_cast<uint4 *>(p)[i] = w16[i];
        } else if constexpr (BYTES == 8) {
            *reinterpret_cast<uint2 *>(p) = w8;
        } else {
            *p = e[0];
        }
    }
};

// Rows of 16-byte words: an item is 16 bytes of the output. Bound by memory:
// 8192 rows of 4096 bf16 in 13.6 us, to fp32 27.6 us. I: a type that counts all
// items.
template <typename S, typename D, typename I>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_kernel(const S *table, long long ldt, const int *ids, D *d, long long ldd, unsigned items, I all, int V, float scale)
{
    constexpr int VEC = 16 / static_cast<int>(sizeof(D));
    grid_start();
    const I first = static_cast<I>(blockIdx.x) * (kEmbedThreads * kEmbedItems) + threadIdx.x;
    Vector<S, VEC> v[kEmbedItems];
    I row[kEmbedItems];
    unsigned col[kEmbedItems];
    int id[kEmbedItems];
#pragma unroll
    for (int i = 0; i < kEmbedItems; ++i) {
        const I at = first + i * kEmbedThreads;
        row[i] = at / items;
        col[i] = static_cast<unsigned>(at - row[i] * items) * VEC;
        id[i] = at < all ? ids[row[i]] : -1;
    }
#pragma unroll
    for (int i = 0; i < kEmbedItems; ++i) {
        if (static_cast<unsigned>(id[i]) < static_cast<unsigned>(V)) {
            v[i].load(table + id[i] * ldt + col[i]);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                v[i].e[j] = from_float<S>(0.0f);
        }
    }
#pragma unroll
    for (int i = 0; i < kEmbedItems; ++i) {
        if (first + i * kEmbedThreads >= all)
            return;
        Vector<D, VEC> o;
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            o.e[j] = from_float<D>(static_cast<unsigned>(id[i]) < static_cast<unsigned>(V) ? to_float(v[i].e[j]) * scale : 0.0f);
        o.store(d + static_cast<long long>(row[i]) * ldd + col[i]);
    }
}

// Other rows, by single elements side by side: the block's x threads walk a row.
template <typename S, typename D>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_narrow_kernel(const S *table, long long ldt, const int *ids, D *d, long long ldd, long long T, int N, int V, float scale)
{
    const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    grid_start();
    if (t >= T)
        return;
    const int id = ids[t];
    const bool have = static_cast<unsigned>(id) < static_cast<unsigned>(V);
    const S *from = table + (have ? id : 0) * ldt;
    D *to = d + t * ldd;
    const int step = static_cast<int>(blockDim.x);
    for (int c = threadIdx.x; c < N; c += 8 * step) {
        float v[8];
        load8<S, false>(from, c, step, have ? N : 0, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] *= scale;
        store8<D, false>(to, c, step, N, v);
    }
}

// ---------------------------------------------------------------- order by id

constexpr int kSortWarps = 16;
constexpr int kSortMaxBins = 512;
constexpr int kSortPart = 2048;      // entries of a block
constexpr int kSortMaxBlocks = 128;
constexpr int kSortBatch = 4;        // entries a lane loads at a time

// One digit of the ids. The first pass reads the caller's ids and drops those
// outside 0..V-1, later ones the entries that the pass before handed out.
struct SortPass {
    const int *ids;
    const int *tokens;  // null: an entry's own place
    int *ids_out, *tokens_out;
    long long n;        // of the first pass
    int *kept;          // entries that are left after it; behind it a counter for the sums, which starts at 0
    int *counts;        // [block][bins]
    int V, shift, bits, bins, blocks;
    bool first;
    // Blocks past the sort's own write a share of the table's zeros meanwhile:
    // units lo .. hi - 1 of 16 bytes (or 2, where rows are not whole 16-byte
    // words), `row` of them a row, `ld` from one row to the next.
    void *zeros;
    bool wide;
    long long ld, row, lo, hi;
};

struct SortPlan {
    int passes, bits, blocks;
};

SortPlan sort_plan(int64_t T, int64_t V)
{
    int bits = 1;
    while ((static_cast<int64_t>(1) << bits) < V)
        ++bits;
    SortPlan p;
    p.passes = (bits + 8) / 9;
    p.bits = (bits + p.passes - 1) / p.passes;
    p.blocks = static_cast<int>(std::min<int64_t>(kSortMaxBlocks, (T + kSortPart - 1) / kSortPart));
    return p;
}

// (By units of 2 bytes, where rows are odd, it is no slower: 131072 rows of 2047
// bf16 in 88 us, of 2048 in 86.)
template <typename U>
__device__ __forceinline__ void write_zeros(U *d, long long ld, long long row, long long lo, long long hi, int thread, int threads)
{
    const U zero = {};
    long long i = lo + thread;
    if (ld == row) {
#pragma unroll 8
        for (; i < hi; i += threads)
            d[i] = zero;
        return;
    }
    for (; i < hi; i += threads)
        d[i / row * ld + i % row] = zero;
}

// True for a block that has written zeros and is done.
__device__ __forceinline__ bool sort_zeros(const SortPass &p)
{
    const int block = static_cast<int>(blockIdx.x) - p.blocks;
    if (block < 0)
        return false;
    const int threads = (static_cast<int>(gridDim.x) - p.blocks) * static_cast<int>(blockDim.x);
    const int thread = block * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
    if (p.wide)
        write_zeros(static_cast<uint4 *>(p.zeros), p.ld, p.row, p.lo, p.hi, thread, threads);
    else
        write_zeros(static_cast<uint16_t *>(p.zeros), p.ld, p.row, p.lo, p.hi, thread, threads);
    return true;
}

__device__ __forceinline__ void sort_load(const SortPass &p, long long i, long long end, int (&id)[kSortBatch])
{
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u)
        id[u] = i + 32 * u < end ? __ldcg(p.ids + i + 32 * u) : -1;
    if (p.first) {
#pragma unroll
        for (int u = 0; u < kSortBatch; ++u)
            if (static_cast<unsigned>(id[u]) >= static_cast<unsigned>(p.V))
                id[u] = -1;
    }
}

__device__ __forceinline__ int sort_digit(const SortPass &p, int id) { return (id >> p.shift) & (p.bins - 1); }

// The lanes that have this lane's digit: a ballot for each of its bits, which is
// quicker than a match over the warp's 32 values.
__device__ __forceinline__ unsigned sort_peers(int digit, int bits, bool valid)
{
    unsigned same = __ballot_sync(0xffffffffu, valid);
    for (int i = 0; i < bits; ++i) {
        const bool set = (digit >> i) & 1;
        const unsigned with = __ballot_sync(0xffffffffu, set);
        same &= set ? with : ~with;
    }
    return same;
}

// Entries of one warp: run `warp` of part `block`, whole steps of 32.
struct SortRun {
    long long lo, hi;
};

__device__ __forceinline__ SortRun sort_run(const SortPass &p, int warp)
{
    const long long n = p.first ? p.n : __ldcg(p.kept);
    const long long part = (n + p.blocks - 1) / p.blocks;
    const long long lo = min(blockIdx.x * part, n), hi = min(lo + part, n);
    const long long run = ((hi - lo + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    SortRun r;
    r.lo = min(lo + warp * run, hi);
    r.hi = min(r.lo + run, hi);
    return r;
}

__device__ void sort_histogram(const SortPass &p, const SortRun &r, int lane, int *hist)
{
    for (long long i0 = r.lo; i0 < r.hi; i0 += 32 * kSortBatch) {
        int id[kSortBatch];
        sort_load(p, i0 + lane, r.hi, id);
#pragma unroll
        for (int u = 0; u < kSortBatch; ++u)
            if (id[u] >= 0)
                atomicAdd(&hist[sort_digit(p, id[u])], 1);  // a count: the order of the additions does not show
    }
}

__global__ void __launch_bounds__(32 * kSortWarps) sort_count_kernel(const SortPass p)
{
    __shared__ int hist[kSortMaxBins];
    for (int b = threadIdx.x; b < p.bins; b += blockDim.x)
        hist[b] = 0;
    grid_start();
    if (sort_zeros(p))
        return;
    __syncthreads();
    sort_histogram(p, sort_run(p, threadIdx.x >> 5), threadIdx.x & 31, hist);
    __syncthreads();
    for (int b = threadIdx.x; b < p.bins; b += blockDim.x)
        p.counts[static_cast<long long>(blockIdx.x) * p.bins + b] = hist[b];
}

// Hands out the entries of one pass: `hist` holds kSortWarps x bins counts,
// `start` and `before` a value for each bin.
__device__ void sort_scatter(const SortPass &p, int *hist, int *start, int *before)
{
    __shared__ int warp_total[kSortWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bins = p.bins;
    for (int i = tid; i < (kSortWarps + 2) * bins; i += blockDim.x)
        hist[i] = 0;  // start and before lie behind it
    __syncthreads();
    const SortRun r = sort_run(p, warp);
    sort_histogram(p, r, lane, hist + warp * bins);
    __syncthreads();
    const int lanes = max(1, static_cast<int>(blockDim.x) / bins);
    for (int i = tid; i < bins * lanes; i += blockDim.x) {
        const int b = i % bins;
        int total = 0, prior = 0;
#pragma unroll 8
        for (int k = i / bins; k < p.blocks; k += lanes) {
            const int c = __ldcg(p.counts + static_cast<long long>(k) * bins + b);
            total += c;
            prior += k < static_cast<int>(blockIdx.x) ? c : 0;
        }
        atomicAdd(&start[b], total);
        atomicAdd(&before[b], prior);
    }
    __syncthreads();
    // exclusive scan of the totals: a bin for each thread (there are at most as many)
    const int mine = tid < bins ? start[tid] : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        warp_total[warp] = incl;
    __syncthreads();
    int at = incl - mine, kept = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        at += w < warp ? warp_total[w] : 0;
        kept += warp_total[w];
    }
    if (p.first && blockIdx.x == 0 && tid == 0) {
        p.kept[0] = kept;
        p.kept[1] = 0;
    }
    // first place of each warp's entries of each bin
    if (tid < bins) {
        at += before[tid];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int n = hist[w * bins + tid];
            hist[w * bins + tid] = at;
            at += n;
        }
    }
    __syncthreads();
    int *next = hist + warp * bins;
    for (long long i0 = r.lo; i0 < r.hi; i0 += 32 * kSortBatch) {
        int id[kSortBatch];
        sort_load(p, i0 + lane, r.hi, id);
#pragma unroll
        for (int u = 0; u < kSortBatch; ++u) {
            const long long i = i0 + 32 * u + lane;
            const int b = sort_digit(p, id[u]);
            const unsigned same = sort_peers(b, p.bits, id[u] >= 0);
            int place = -1;
            if (id[u] >= 0)
                place = next[b] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (id[u] >= 0 && (same >> lane) == 1u)  // the last of its bin moves the count on
                next[b] = place + 1;
            __syncwarp();
            if (place >= 0) {
                p.ids_out[place] = id[u];
                p.tokens_out[place] = p.tokens ? __ldcg(p.tokens + i) : static_cast<int>(i);
            }
        }
    }
}

__global__ void __launch_bounds__(32 * kSortWarps) sort_scatter_kernel(const SortPass p)
{
    extern __shared__ int sort_smem[];
    grid_start();
    if (sort_zeros(p))
        return;
    sort_scatter(p, sort_smem, sort_smem + kSortWarps * p.bins, sort_smem + (kSortWarps + 1) * p.bins);
}

// Up to 16384 tokens: one launch. Each block has a range of ids and looks through
// all of the list (which L2 holds) for those of its range: it counts the ids
// below the range, which is where its own begin in the order, and its own by
// warp and id; then it hands them out, each warp its run of the list. Of a
// gradient that is written whole, warps of their own zero its range's rows
// meanwhile. Blocks need nothing of one another. (A counting sort by digits
// takes four launches that wait for one another; by one block of 32 warps it
// took 35 us for 16384 tokens of 32768 ids.) Every block reads all of the list, so
// that more tokens are better sorted by digits: rows of 64 added into 32768 ids
// 4096 tokens 14.8 us by ranges and 25.7 by digits, 16384 27.8 and 36.7, 20000 31.4
// and 38.0, 32768 41.5 and 40.1, 65536 70.8 and 51.2; into 1000 ids 20000 32.9 and
// 31.2; rows of 2048 written whole 16384 52.7 and 63.9, 32768 80.1 and 79.9, 65536
// 134.5 and 119.5. The two cross between 20000 and 32768 tokens.
constexpr int kRangeWarps = 16;
constexpr int kRangeBatch = 8;          // entries a lane has in flight
constexpr int kRangeBlocks = 152;       // at least: one for each SM of the GPU this is built for
constexpr int kRangeMostIds = 1024;     // of a block
constexpr int kRangeMostBlocks = 1024;
constexpr int64_t kRangeMostTokens = 16384;
constexpr int kZeroWarps = 16;          // of a block that writes its range's zeros meanwhile

inline bool sort_by_range(int64_t T, int64_t V) { return T <= kRangeMostTokens && V <= static_cast<int64_t>(kRangeMostIds) * kRangeMostBlocks; }

struct RangePass {
    const int *ids;
    int *ids_out, *tokens_out, *kept;
    int T, V, per;  // ids of a block
    void *zeros;    // the table, or null: rows as in SortPass
    bool wide;
    long long ld, row, all;
};

// The sorting warps' barrier.
__device__ __forceinline__ void range_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kRangeWarps) : "memory"); }

__global__ void __launch_bounds__(32 * (kRangeWarps + kZeroWarps)) sort_range_kernel(const RangePass p)
{
    extern __shared__ int range_smem[];
    __shared__ int warp_total[kRangeWarps], below_all, all_kept;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *hist = range_smem;  // [warp][id of the range]
    const int first = static_cast<int>(blockIdx.x) * p.per, n = min(p.per, p.V - first);
    if (warp >= kRangeWarps) {
        grid_start();
        // all blocks walk the table side by side
        const int thread = tid - 32 * kRangeWarps + static_cast<int>(blockIdx.x) * (32 * kZeroWarps), threads = static_cast<int>(gridDim.x) * (32 * kZeroWarps);
        if (p.wide)
            write_zeros(static_cast<uint4 *>(p.zeros), p.ld, p.row, 0, p.all, thread, threads);
        else
            write_zeros(static_cast<uint16_t *>(p.zeros), p.ld, p.row, 0, p.all, thread, threads);
        return;
    }
    for (int i = tid; i < kRangeWarps * n; i += 32 * kRangeWarps)
        hist[i] = 0;
    if (tid == 0)
        below_all = all_kept = 0;
    grid_start();
    range_sync();
    // the warp's run of the list, whole steps of 32
    const int run = ((p.T + kRangeWarps - 1) / kRangeWarps + 31) / 32 * 32;
    const int lo = min(warp * run, p.T), hi = min(lo + run, p.T);
    int *mine = hist + warp * n;
    int below = 0, kept = 0;
    for (int i0 = lo; i0 < hi; i0 += 32 * kRangeBatch) {
        int id[kRangeBatch];
#pragma unroll
        for (int u = 0; u < kRangeBatch; ++u)
            id[u] = i0 + 32 * u + lane < hi ? __ldcg(p.ids + i0 + 32 * u + lane) : -1;
#pragma unroll
        for (int u = 0; u < kRangeBatch; ++u) {
            if (static_cast<unsigned>(id[u]) < static_cast<unsigned>(p.V)) {
                ++kept;
                below += id[u] < first;
                if (static_cast<unsigned>(id[u] - first) < static_cast<unsigned>(n))
                    atomicAdd(&mine[id[u] - first], 1);  // a count: the order of the additions does not show
            }
        }
    }
    below = __reduce_add_sync(0xffffffffu, below);
    kept = __reduce_add_sync(0xffffffffu, kept);
    if (lane == 0) {
        atomicAdd(&below_all, below);
        atomicAdd(&all_kept, kept);
    }
    range_sync();
    if (blockIdx.x == 0 && tid == 0) {
        p.kept[0] = all_kept;
        p.kept[1] = 0;
    }
    // where each id's entries begin, two ids a thread, and each warp's of them
    static_assert(kRangeMostIds <= 2 * 32 * kRangeWarps, "two ids a thread");
    int total[2] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (2 * tid + k < n) {
#pragma unroll
            for (int w = 0; w < kRangeWarps; ++w)
                total[k] += hist[w * n + 2 * tid + k];
        }
    const int sum = total[0] + total[1];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        warp_total[warp] = incl;
    range_sync();
    int at = below_all + incl - sum, own = 0;
#pragma unroll
    for (int w = 0; w < kRangeWarps; ++w) {
        at += w < warp ? warp_total[w] : 0;
        own += warp_total[w];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (2 * tid + k < n) {
            const int id = 2 * tid + k;
#pragma unroll
            for (int w = 0; w < kRangeWarps; ++w) {
                const int c = hist[w * n + id];
                hist[w * n + id] = at;
                at += c;
            }
        }
    range_sync();
    if (own == 0)
        return;
    for (int i0 = lo; i0 < hi; i0 += 32 * kRangeBatch) {
        int id[kRangeBatch];
#pragma unroll
        for (int u = 0; u < kRangeBatch; ++u)
            id[u] = i0 + 32 * u + lane < hi ? __ldcg(p.ids + i0 + 32 * u + lane) - first : -1;
#pragma unroll
        for (int u = 0; u < kRangeBatch; ++u) {
            unsigned left = __ballot_sync(0xffffffffu, static_cast<unsigned>(id[u]) < static_cast<unsigned>(n));
            while (left) {  // an id at a time: a block has few of 32 entries, or the same ones often
                const int who = __shfl_sync(0xffffffffu, id[u], __ffs(left) - 1);
                const unsigned same = __ballot_sync(0xffffffffu, id[u] == who) & left;
                const int place = mine[who];
                if (id[u] == who) {
                    const int to = place + __popc(same & ((1u << lane) - 1u));
                    p.ids_out[to] = who + first;
                    p.tokens_out[to] = i0 + 32 * u + lane;
                }
                __syncwarp();
                if (lane == 0)
                    mine[who] = place + __popc(same);
                __syncwarp();
                left &= ~same;
            }
        }
    }
}

std::atomic<uint64_t> range_attribute_set[2] = {{0}, {0}};

// ---------------------------------------------------------------- sums

constexpr int kMaxChunk = 32;       // sorted entries of a block at most
constexpr int kSumThreads = 128;    // of eight columns each
constexpr int kSumColumns = 8 * kSumThreads;
constexpr int kSumBlocks = 608;     // four for each SM of the GPU this is built for
constexpr int kJoinBlocks = 152;   // one for each
constexpr int kJoinGroups = 4;      // of kSumThreads threads in a block that joins chunks
constexpr int kJoinAlone = 8;       // parts that one group joins by itself

struct SumParams {
    long long T;
    const int *ids, *tokens, *kept;
    int *crossing, *crossings;  // the chunks in which a run begins that passes their end, in any order, and their number
    long long lddd, ldt;
    int N, accumulate, col_blocks, chunk;
    float scale;
    float *parts;  // [2 * chunks][N8]: a chunk's first run where it began before, its last where it goes on
    long long ld_parts;
};

// Eight elements of a row as load8 takes them, not yet widened.
template <typename T>
struct Eight {
    union {
        uint4 w[sizeof(T) / 2];
        T e[8];
    };
    __device__ __forceinline__ Eight() {}
    template <bool WIDE>
    __device__ __forceinline__ void load(const T *p, int at, int step, int n)
    {
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
                w[i] = at < n ? reinterpret_cast<const uint4 *>(p + at)[i] : make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                e[i] = at + i * step < n ? p[at + i * step] : from_float<T>(0.0f);
        }
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = to_float(e[i]);
    }
};

// dtable[id] = scale * sum (+ what it holds)
template <typename W, bool WIDE>
__device__ __forceinline__ void finish_row(W *row, int c, int N, float (&acc)[8], float scale, int accumulate)
{
    float old[8];
    if (accumulate)
        load8<W, WIDE>(row, c, kSumThreads, N, old);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        acc[i] = accumulate ? fmaf(acc[i], scale, old[i]) : acc[i] * scale;
    store8<W, WIDE>(row, c, kSumThreads, N, acc);
}

// Sums the runs of one chunk: a block has 1024 columns of it. ADD: to what the
// table holds, which is asked for with the last row of each run.
template <typename D, typename W, bool WIDE, bool ADD>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const D *dd, W *dtable, const SumParams p)
{
    constexpr int ROWS = WIDE && sizeof(D) == 2 ? 8 : 4;  // in flight: as many as registers hold
    __shared__ int ids[kMaxChunk + 2];                    // with the entries before and behind
    __shared__ long long rows[kMaxChunk];
    const int tid = threadIdx.x;
    const long long chunk = blockIdx.x / p.col_blocks;
    const int col_block = static_cast<int>(blockIdx.x - chunk * p.col_blocks);
    const int c = col_block * kSumColumns + (WIDE ? 8 : 1) * tid;
    grid_start();
    const long long lo = chunk * p.chunk, i = lo + tid - 1;
    // asked for together; what lies past the kept entries is not looked at
    const bool near = tid < p.chunk + 2 && i >= 0 && i < p.T;
    const int id = near ? __ldcg(p.ids + i) : -1, token = near ? __ldcg(p.tokens + i) : 0;
    const long long kept = __ldcg(p.kept);
    if (lo >= kept)
        return;
    const int n = static_cast<int>(min(kept - lo, static_cast<long long>(p.chunk)));
    if (tid < p.chunk + 2)
        ids[tid] = i < kept ? id : -1;
    // places past the last name the first row, which is not added for them
    if (tid > 0 && tid <= p.chunk)
        rows[tid - 1] = (tid <= n ? token : 0) * p.lddd;
    __syncthreads();
    if (c >= p.N)
        return;
    float acc[8] = {};
    int run = ids[1];
    bool before = ids[0] == run;  // the run began in an earlier chunk
    auto part = [&](int which) { store8<float, WIDE>(p.parts + (2 * chunk + which) * p.ld_parts, c, kSumThreads, p.N, acc); };
    for (int j0 = 0; j0 < n; j0 += ROWS) {
        Eight<D> raw[ROWS];
        Eight<W> old[ADD ? ROWS : 1];
#pragma unroll
        for (int u = 0; u < ROWS; ++u)
            raw[u].template load<WIDE>(dd + rows[j0 + u], c, kSumThreads, p.N);
        if constexpr (ADD) {
#pragma unroll
            for (int u = 0; u < ROWS; ++u)
                if (j0 + u < n && ids[1 + j0 + u] != ids[2 + j0 + u])
                    old[u].template load<WIDE>(dtable + ids[1 + j0 + u] * p.ldt, c, kSumThreads, p.N);
        }
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            const int j = j0 + u;
            if (j >= n)
                break;
            float v[8];
            raw[u].values(v);
            if (ids[1 + j] != run) {
                run = ids[1 + j];
                before = false;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    acc[k] = v[k];
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    acc[k] += v[k];
            }
            if (ids[2 + j] != run) {  // the run ends here
                if (before) {
                    part(0);
                } else {
                    if constexpr (ADD)
                        old[u].values(v);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        acc[k] = ADD ? fmaf(acc[k], p.scale, v[k]) : acc[k] * p.scale;
                    store8<W, WIDE>(dtable + run * p.ldt, c, kSumThreads, p.N, acc);
                }
            }
        }
    }
    if (ids[n + 1] == run) {  // it goes on behind the chunk
        part(before ? 0 : 1);
        if (!before && col_block == 0 && tid == 0)
            p.crossing[atomicAdd(p.crossings, 1)] = static_cast<int>(chunk);
    }
}

// Joins the parts of each run that passes a chunk's end, in the order of the
// chunks. A group of threads takes a run (1024 columns of it) of the list, whose
// order does not show, as its sums' orders are its own; where it has many
// parts, all groups of the block take equal shares of it.
template <typename W, bool WIDE>
__global__ void __launch_bounds__(kSumThreads * kJoinGroups) embed_join_kernel(W *dtable, const SumParams p)
{
    __shared__ float share_sums[kJoinGroups - 1][8][kSumThreads];
    __shared__ int long_chunk[kJoinGroups], long_cols[kJoinGroups];
    __shared__ long long long_more[kJoinGroups];
    const int tid = threadIdx.x, group = threadIdx.y, lane = tid & 31;
    grid_start();
    const int items = __ldcg(p.crossings) * p.col_blocks;
    for (int first = blockIdx.x * kJoinGroups; first < items; first += kJoinBlocks * kJoinGroups) {
        const int item = first + group;
        if (tid == 0)
            long_more[group] = 0;
        __syncthreads();
        if (item < items) {
            const int chunk = __ldcg(p.crossing + item / p.col_blocks), col_block = item % p.col_blocks;
            const long long next = (chunk + 1ll) * p.chunk, kept = __ldcg(p.kept);
            const long long all = (kept - next + p.chunk - 1) / p.chunk;  // chunks behind this one
            const int run = __ldcg(p.ids + next);
            // those that begin with the run: each warp narrows them down, 32 at
            // a time at first: the first `more` do, those from `most` on do not
            long long more = 0, most = all;
            for (long long step = 1; more < most; step = (most - more + 31) / 32) {
                const long long at = more + lane * step;
                const unsigned yes = __ballot_sync(0xffffffffu, at < most && __ldcg(p.ids + next + min(at, most - 1) * p.chunk) == run);
                const int hits = __popc(yes);  // of ascending places: the first ones
                if (hits < 32)
                    most = min(most, more + hits * step);
                if (hits > 0)
                    more += (hits - 1) * step + 1;
            }
            if (more > kJoinAlone) {
                if (tid == 0) {
                    long_chunk[group] = chunk;
                    long_cols[group] = col_block;
                    long_more[group] = more;
                }
            } else {
                const int c = col_block * kSumColumns + (WIDE ? 8 : 1) * tid;
                float acc[8], v[kJoinAlone][8];
                load8<float, WIDE>(p.parts + (2ll * chunk + 1) * p.ld_parts, c, kSumThreads, p.N, acc);
#pragma unroll
                for (int k = 0; k < kJoinAlone; ++k)
                    load8<float, WIDE>(p.parts + 2 * (chunk + 1 + (k < more ? k : 0)) * p.ld_parts, c, kSumThreads, k < more ? p.N : 0, v[k]);
#pragma unroll
                for (int k = 0; k < kJoinAlone; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        acc[j] += v[k][j];
                if (c < p.N)
                    finish_row<W, WIDE>(dtable + run * p.ldt, c, p.N, acc, p.scale, p.accumulate);
            }
        }
        __syncthreads();
        for (int g = 0; g < kJoinGroups; ++g) {
            const long long more = long_more[g];
            if (more == 0)
                continue;
            const long long chunk = long_chunk[g];
            const int c = long_cols[g] * kSumColumns + (WIDE ? 8 : 1) * tid;
            const long long share = (more + kJoinGroups - 1) / kJoinGroups;
            const long long from = chunk + 1 + group * share, to = min(from + share, chunk + 1 + more);
            float acc[8] = {};
            if (group == 0)
                load8<float, WIDE>(p.parts + (2 * chunk + 1) * p.ld_parts, c, kSumThreads, p.N, acc);
            for (long long k = from; k < to; k += kJoinAlone) {
                float v[kJoinAlone][8];
#pragma unroll
                for (int u = 0; u < kJoinAlone; ++u)
                    load8<float, WIDE>(p.parts + 2 * min(k + u, to - 1) * p.ld_parts, c, kSumThreads, k + u < to ? p.N : 0, v[u]);
#pragma unroll
                for (int u = 0; u < kJoinAlone; ++u)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        acc[j] += v[u][j];
            }
            if (group > 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    share_sums[group - 1][j][tid] = acc[j];
            }
            __syncthreads();
            if (group == 0 && c < p.N) {
#pragma unroll
                for (int k = 0; k < kJoinGroups - 1; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        acc[j] += share_sums[k][j][tid];
                finish_row<W, WIDE>(dtable + __ldcg(p.ids + (chunk + 1) * p.chunk) * p.ldt, c, p.N, acc, p.scale, p.accumulate);
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------- zeros

__global__ void __launch_bounds__(512) embed_zero_kernel(SortPass p)
{
    grid_start();
    sort_zeros(p);
}

struct EmbedPlan {
    SortPlan sort;
    int chunk;
    int64_t chunks;
    size_t kept, crossing, counts, ids_a, tokens_a, ids_b, tokens_b, parts, bytes;  // offsets
    int64_t ld_parts;
};

int64_t column_blocks(int64_t N) { return (N + kSumColumns - 1) / kSumColumns; }

// Entries of a chunk: as many as leave the SMs four blocks each.
int chunk_of(int64_t T, int64_t N)
{
    const int64_t rows = T * column_blocks(N);
    return rows >= 32 * kSumBlocks ? 32 : rows >= 16 * kSumBlocks ? 16 : 8;
}

EmbedPlan embed_plan(int64_t T, int64_t N, int64_t V)
{
    EmbedPlan e = {};
    e.sort = sort_plan(T, V);
    e.chunk = chunk_of(T, N);
    e.chunks = (T + e.chunk - 1) / e.chunk;
    e.ld_parts = (N + 7) / 8 * 8;
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t o = at;
        at += static_cast<size_t>((bytes + 255) / 256 * 256);
        return o;
    };
    e.kept = take(8);
    e.crossing = take(4 * e.chunks);
    const bool range = sort_by_range(T, V);
    e.counts = take(range ? 0 : static_cast<int64_t>(e.sort.blocks) * 4 << e.sort.bits);
    e.ids_a = take(4 * T);
    e.tokens_a = take(4 * T);
    e.ids_b = take(!range && e.sort.passes > 1 ? 4 * T : 0);
    e.tokens_b = take(!range && e.sort.passes > 1 ? 4 * T : 0);
    e.parts = take(e.chunks > 1 ? 2 * e.chunks * e.ld_parts * 4 : 0);
    e.bytes = at;
    return e;
}

// Room for T tokens and for fewer. With chunks of one length more tokens need
// more; where chunks get longer there are fewer of them, so that the most tokens
// of each shorter length may need more than T.
size_t embed_bytes(int64_t T, int64_t N, int64_t V)
{
    size_t most = embed_plan(T, N, V).bytes;
    for (int chunk = 16; chunk <= chunk_of(T, N); chunk *= 2) {
        const int64_t before = (chunk * static_cast<int64_t>(kSumBlocks) - 1) / column_blocks(N);
        if (before > 0)
            most = std::max(most, embed_plan(before, N, V).bytes);
    }
    return most;
}

constexpr int kZeroBlocks = 304;  // beside the sort's

gemm_status_t launch_sort(const EmbedPlan &e, SortPass p, int64_t T, int64_t V, const int32_t *ids, uint8_t *ws, cudaStream_t st)
{
    int *at[4] = {reinterpret_cast<int *>(ws + e.ids_a), reinterpret_cast<int *>(ws + e.tokens_a), reinterpret_cast<int *>(ws + e.ids_b),
                  reinterpret_cast<int *>(ws + e.tokens_b)};
    p.ids = ids;
    p.n = T;
    p.kept = reinterpret_cast<int *>(ws + e.kept);
    p.counts = reinterpret_cast<int *>(ws + e.counts);
    p.V = static_cast<int>(V);
    p.bits = e.sort.bits;
    p.bins = 1 << e.sort.bits;
    p.blocks = e.sort.blocks;
    const int64_t zeros = p.hi;  // of the whole table
    const unsigned grid = static_cast<unsigned>(p.blocks + (zeros > 0 ? std::min<int64_t>(kZeroBlocks, (zeros + 511) / 512) : 0));
    const size_t smem = static_cast<size_t>(kSortWarps + 2) * p.bins * sizeof(int);
    int launch = 0;
    auto share = [&]() {  // equal shares of the zeros for every launch
        p.lo = zeros * launch / (2 * e.sort.passes);
        p.hi = zeros * (launch + 1) / (2 * e.sort.passes);
        ++launch;
    };
    for (int i = 0; i < e.sort.passes; ++i) {
        p.first = i == 0;
        p.shift = i * e.sort.bits;
        if (i > 0) {
            p.ids = p.ids_out;
            p.tokens = p.tokens_out;
        }
        const int to = (e.sort.passes - i) % 2 ? 0 : 2;  // the last pass writes to a
        p.ids_out = at[to];
        p.tokens_out = at[to + 1];
        share();
        gemm_status_t s = host_launch(sort_count_kernel, grid, 32 * kSortWarps, 0, st, 0, p);
        share();
        if (s != GEMM_OK || (s = host_launch(sort_scatter_kernel, grid, 32 * kSortWarps, smem, st, 0, p)) != GEMM_OK)
            return s;
    }
    return GEMM_OK;
}

bool wide_rows(const void *p, int64_t ld, int64_t N, int es) { return N % 8 == 0 && aligned_to(p, 16) && ld * es % 16 == 0; }

// What both calls check of their shape, the table and the rows.
gemm_status_t check_embed(int64_t T, int64_t N, int64_t V, const int32_t *ids, const void *table, int t_type, int64_t ldt, float scale,
                          const void *D, int d_type, int64_t ldd)
{
    if (!valid_size(T) || !valid_size(N) || !valid_size(V) || !valid_type(t_type) || !valid_type(d_type) || !std::isfinite(scale))
        return GEMM_ERR_INVALID_ARG;
    const int et = type_bytes(t_type), ed = type_bytes(d_type);
    if ((T > 0 && N > 0 && (!ids || !D || (V > 0 && !table))) || ldt < N || ldd < N || !valid_stride(ldt, et) || !valid_stride(ldd, ed))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(ids, 4) || !aligned_to(table, et) || !aligned_to(D, ed))
        return GEMM_ERR_ALIGNMENT;
    if (!countable(T) || !countable(N) || !countable(V))
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

}  // namespace

// ---------------------------------------------------------------- C ABI

extern "C" {

gemm_status_t gemm_embed(int64_t T, int64_t N, int64_t V, const int32_t *ids, const void *table, gemm_out_t t_type, int64_t ldt, float scale,
                         void *D, gemm_out_t d_type, int64_t ldd, gemm_stream_t stream)
{
    const gemm_status_t s = check_embed(T, N, V, ids, table, t_type, ldt, scale, D, d_type, ldd);
    if (s != GEMM_OK || T == 0 || N == 0)
        return s;
    const bool wide = wide_rows(table, ldt, N, type_bytes(t_type)) && wide_rows(D, ldd, N, type_bytes(d_type));
    const int64_t items = N * type_bytes(d_type) / 16, all = T * items, block = kEmbedThreads * kEmbedItems;
    const int64_t blocks = (all + block - 1) / block;
    // threads of a narrow row, eight columns each, and rows of a block
    const int x = static_cast<int>(std::min<int64_t>(kEmbedThreads, ((N + 7) / 8 + 31) / 32 * 32)), y = kEmbedThreads / x;
    if (wide && blocks > kSizeLimit)
        return GEMM_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return with_type(t_type, [&](auto ttag) {
        using S = decltype(ttag);
        return with_type(d_type, [&](auto dtag) {
            using D_ = decltype(dtag);
            const S *from = static_cast<const S *>(table);
            D_ *to = static_cast<D_ *>(D);
            const int v = static_cast<int>(V);
            if (!wide)
                return host_launch(embed_narrow_kernel<S, D_>, static_cast<unsigned>((T + y - 1) / y), dim3(x, y), 0, st, 0, from, ldt, ids, to, ldd,
                                   T, static_cast<int>(N), v, scale);
            const unsigned grid = static_cast<unsigned>(blocks), row = static_cast<unsigned>(items);
            if (blocks * block <= UINT32_MAX)  // items are counted in 32 bits
                return host_launch(embed_kernel<S, D_, unsigned>, grid, kEmbedThreads, 0, st, 0, from, ldt, ids, to, ldd, row, all, v, scale);
            return host_launch(embed_kernel<S, D_, unsigned long long>, grid, kEmbedThreads, 0, st, 0, from, ldt, ids, to, ldd, row, all, v, scale);
        });
    });
}

size_t gemm_embed_backward_workspace_size(int64_t T, int64_t N, int64_t V)
{
    if (T < 1 || N < 1 || V < 1 || !countable(T) || !countable(N) || !countable(V))
        return 0;
    return embed_bytes(T, N, V);
}

gemm_status_t gemm_embed_backward(int64_t T, int64_t N, int64_t V, const int32_t *ids, const void *dD, gemm_out_t d_type, int64_t lddd,
                                  float scale, void *dtable, gemm_out_t t_type, int64_t lddt, int accumulate, void *workspace,
                                  size_t workspace_bytes, gemm_stream_t stream)
{
    gemm_status_t s = check_embed(T, N, V, ids, dtable, t_type, lddt, scale, dD, d_type, lddd);
    if (s != GEMM_OK || N == 0 || V == 0)
        return s;
    if (!dtable)
        return GEMM_ERR_INVALID_ARG;
    const EmbedPlan e = embed_plan(std::max<int64_t>(T, 1), N, V);
    const size_t need = T > 0 ? e.bytes : 0;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return GEMM_ERR_INVALID_ARG;
    if (need > 0 && !aligned_to(workspace, 256))
        return GEMM_ERR_ALIGNMENT;
    const int64_t col_blocks = column_blocks(N);
    if (col_blocks * e.chunks > kSizeLimit)
        return GEMM_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int et = type_bytes(t_type);
    SortPass sort = {};
    if (!accumulate) {
        sort.wide = aligned_to(dtable, 16) && (N * et % 16 == 0) && (lddt * et % 16 == 0);
        const int64_t unit = sort.wide ? 16 : 2;
        sort.zeros = dtable;
        sort.row = N * et / unit;
        sort.ld = lddt * et / unit;
        sort.hi = V * sort.row;
    }
    if (T == 0)
        return accumulate ? GEMM_OK : host_launch(embed_zero_kernel, 2u * kZeroBlocks, 512, 0, st, 0, sort);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (sort_by_range(T, V)) {
        RangePass r = {};
        r.ids = ids;
        r.ids_out = reinterpret_cast<int *>(ws + e.ids_a);
        r.tokens_out = reinterpret_cast<int *>(ws + e.tokens_a);
        r.kept = reinterpret_cast<int *>(ws + e.kept);
        r.T = static_cast<int>(T);
        r.V = static_cast<int>(V);
        r.per = static_cast<int>(std::min<int64_t>(kRangeMostIds, (V + kRangeBlocks - 1) / kRangeBlocks));
        r.zeros = sort.zeros;
        r.wide = sort.wide;
        r.ld = sort.ld;
        r.row = sort.row;
        r.all = sort.hi;
        const size_t smem = static_cast<size_t>(kRangeWarps) * r.per * sizeof(int);
        if (ensure_smem_attribute(sort_range_kernel, kRangeWarps * kRangeMostIds * 4, range_attribute_set) != cudaSuccess)
            return GEMM_ERR_CUDA;
        s = host_launch(sort_range_kernel, static_cast<unsigned>((V + r.per - 1) / r.per), 32 * (kRangeWarps + (accumulate ? 0 : kZeroWarps)), smem, st,
                        0, r);
    } else {
        s = launch_sort(e, sort, T, V, ids, ws, st);
    }
    if (s != GEMM_OK)
        return s;
    SumParams p = {};
    p.T = T;
    p.ids = reinterpret_cast<int *>(ws + e.ids_a);
    p.tokens = reinterpret_cast<int *>(ws + e.tokens_a);
    p.kept = reinterpret_cast<int *>(ws + e.kept);
    p.crossings = reinterpret_cast<int *>(ws + e.kept) + 1;
    p.crossing = reinterpret_cast<int *>(ws + e.crossing);
    p.lddd = lddd;
    p.ldt = lddt;
    p.N = static_cast<int>(N);
    p.accumulate = accumulate != 0;
    p.col_blocks = static_cast<int>(col_blocks);
    p.chunk = e.chunk;
    p.scale = scale;
    p.parts = reinterpret_cast<float *>(ws + e.parts);
    p.ld_parts = e.ld_parts;
    const bool wide = wide_rows(dD, lddd, N, type_bytes(d_type)) && wide_rows(dtable, lddt, N, et);
    const unsigned grid = static_cast<unsigned>(col_blocks * e.chunks);
    return with_type(t_type, [&](auto ttag) {
        using W = decltype(ttag);
        return with_type(d_type, [&](auto dtag) {
            using D = decltype(dtag);
            const D *from = static_cast<const D *>(dD);
            W *to = static_cast<W *>(dtable);
            const auto sums = accumulate ? (wide ? embed_sum_kernel<D, W, true, true> : embed_sum_kernel<D, W, false, true>)
                                         : (wide ? embed_sum_kernel<D, W, true, false> : embed_sum_kernel<D, W, false, false>);
            gemm_status_t r = host_launch(sums, grid, kSumThreads, 0, st, 0, from, to, p);
            if (r != GEMM_OK || e.chunks == 1)
                return r;
            return host_launch(wide ? embed_join_kernel<W, true> : embed_join_kernel<W, false>, kJoinBlocks, dim3(kSumThreads, kJoinGroups), 0, st,
                               0, to, p);
        });
    });
}

}  // extern "C"
