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

// An item is 16 bytes of the output (WIDE: rows of 16-byte words) or a single
// element. Bound by memory. I: a type that counts all items.
template <typename S, typename D, bool WIDE, typename I>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_kernel(const S *table, long long ldt, const int *ids, D *d, long long ldd, unsigned items, I all, int V, float scale)
{
    constexpr int VEC = WIDE ? 16 / static_cast<int>(sizeof(D)) : 1;
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

// ---------------------------------------------------------------- order by id

constexpr int kBlockWarps = 32;
constexpr int kBlockSteps = 16;                             // of 32 entries for each warp
constexpr int kBlockMost = 32 * kBlockWarps * kBlockSteps;  // entries that one block sorts

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
    int *kept;          // entries that are left after it
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
    p.blocks = T <= kBlockMost ? 1 : static_cast<int>(std::min<int64_t>(kSortMaxBlocks, (T + kSortPart - 1) / kSortPart));
    return p;
}

template <typename U>
__device__ __forceinline__ void write_zeros(U *d, long long ld, long long row, long long lo, long long hi, int block, int blocks)
{
    const long long step = static_cast<long long>(blocks) * blockDim.x;
    const U zero = {};
    long long i = lo + static_cast<long long>(block) * blockDim.x + threadIdx.x;
    if (ld == row) {
#pragma unroll 4
        for (; i < hi; i += step)
            d[i] = zero;
        return;
    }
    for (; i < hi; i += step)
        d[i / row * ld + i % row] = zero;
}

// True for a block that has written zeros and is done.
__device__ __forceinline__ bool sort_zeros(const SortPass &p)
{
    const int block = static_cast<int>(blockIdx.x) - p.blocks;
    if (block < 0)
        return false;
    const int blocks = static_cast<int>(gridDim.x) - p.blocks;
    if (p.wide)
        write_zeros(static_cast<uint4 *>(p.zeros), p.ld, p.row, p.lo, p.hi, block, blocks);
    else
        write_zeros(static_cast<uint16_t *>(p.zeros), p.ld, p.row, p.lo, p.hi, block, blocks);
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
// quicker than a match over the warp's 32 values (16384 entries of 15 bits,
// sorted by one block: MATCH_US us by matches).
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
    if (p.first && blockIdx.x == 0 && tid == 0)
        *p.kept = kept;
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

// All passes of a list that one block sorts: the entries are held in registers
// from counting to handing out, and go from pass to pass through shared memory.
// Several launches of more blocks wait longer for one another than they save
// (16384 entries: 30 us by four launches, all but hidden behind 134 MB of zeros
// by this one).
__global__ void __launch_bounds__(32 * kBlockWarps) sort_block_kernel(const SortPass p, int passes, int *ids_out, int *tokens_out)
{
    extern __shared__ int sort_smem[];
    __shared__ int warp_total[kBlockWarps];
    const int bits = p.bits, bins = p.bins, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *hist = sort_smem;                                        // [warp][bin]
    int *list = hist + kBlockWarps * bins;                        // ids between two passes
    uint16_t *places = reinterpret_cast<uint16_t *>(list + p.n);  // and their tokens
    grid_start();
    if (sort_zeros(p))
        return;
    int n = static_cast<int>(p.n), id[kBlockSteps], token[kBlockSteps];
    for (int pass = 0; pass < passes; ++pass) {
        const int steps = (n + 32 * kBlockWarps - 1) / (32 * kBlockWarps), lo = warp * 32 * steps + lane;
#pragma unroll
        for (int u = 0; u < kBlockSteps; ++u) {
            const int i = lo + 32 * u;
            id[u] = -1;
            if (u < steps && i < n) {
                id[u] = pass == 0 ? __ldcg(p.ids + i) : list[i];
                token[u] = pass == 0 ? i : places[i];
            }
        }
        for (int i = tid; i < kBlockWarps * bins; i += 32 * kBlockWarps)
            hist[i] = 0;
        __syncthreads();
        const int shift = pass * bits;
        int *mine = hist + warp * bins;
#pragma unroll
        for (int u = 0; u < kBlockSteps; ++u) {
            if (static_cast<unsigned>(id[u]) >= static_cast<unsigned>(p.V))
                id[u] = -1;
            if (id[u] >= 0)
                atomicAdd(&mine[(id[u] >> shift) & (bins - 1)], 1);  // a count: the order of the additions does not show
        }
        __syncthreads();
        int total = 0;  // of bin tid
        if (tid < bins) {
#pragma unroll 8
            for (int w = 0; w < kBlockWarps; ++w)
                total += hist[w * bins + tid];
        }
        int incl = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += v;
        }
        if (lane == 31)
            warp_total[warp] = incl;
        __syncthreads();
        int at = incl - total, kept = 0;
#pragma unroll 8
        for (int w = 0; w < kBlockWarps; ++w) {
            at += w < warp ? warp_total[w] : 0;
            kept += warp_total[w];
        }
        if (tid < bins) {
#pragma unroll 8
            for (int w = 0; w < kBlockWarps; ++w) {
                const int c = hist[w * bins + tid];
                hist[w * bins + tid] = at;
                at += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kBlockSteps; ++u) {
            if (u < steps) {
                const int b = (id[u] >> shift) & (bins - 1);
                const unsigned same = sort_peers(b, bits, id[u] >= 0);
                int place = -1;
                if (id[u] >= 0)
                    place = mine[b] + __popc(same & ((1u << lane) - 1u));
                __syncwarp();
                if (id[u] >= 0 && (same >> lane) == 1u)  // the last of its bin moves the count on
                    mine[b] = place + 1;
                __syncwarp();
                if (place >= 0) {
                    if (pass == passes - 1) {
                        ids_out[place] = id[u];
                        tokens_out[place] = token[u];
                    } else {
                        list[place] = id[u];
                        places[place] = static_cast<uint16_t>(token[u]);
                    }
                }
            }
        }
        n = kept;
        __syncthreads();
    }
    if (tid == 0)
        *p.kept = n;
}

std::atomic<uint64_t> sort_attribute_set[2] = {{0}, {0}};

// ---------------------------------------------------------------- sums

constexpr int kMaxChunk = 32;       // sorted entries of a block at most
constexpr int kSumThreads = 128;    // of eight columns each
constexpr int kSumColumns = 8 * kSumThreads;
constexpr int kJoinGroups = 4;      // threads that share a column when chunks are joined
constexpr int kSumBlocks = 608;     // four for each SM of the GPU this is built for

struct SumParams {
    const int *ids, *tokens, *kept;
    long long lddd, ldt;
    int N, accumulate, col_blocks, chunk;
    float scale;
    float *parts;  // [2 * chunks][N8]: a chunk's first run where it began before, its last where it goes on
    long long ld_parts;
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

// Sums the runs of one chunk: a block has 1024 columns of it.
template <typename D, typename W, bool WIDE>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const D *dd, W *dtable, const SumParams p)
{
    __shared__ int ids[kMaxChunk + 2], tokens[kMaxChunk];  // with the entries before and behind
    const int tid = threadIdx.x;
    const long long chunk = blockIdx.x / p.col_blocks;
    const int c = static_cast<int>(blockIdx.x - chunk * p.col_blocks) * kSumColumns + (WIDE ? 8 : 1) * tid;
    grid_start();
    const long long kept = __ldcg(p.kept), lo = chunk * p.chunk;
    if (lo >= kept)
        return;
    const int n = static_cast<int>(min(kept - lo, static_cast<long long>(p.chunk)));
    if (tid < p.chunk + 2) {
        const long long i = lo + tid - 1;
        ids[tid] = i >= 0 && i < kept ? __ldcg(p.ids + i) : -1;
        if (tid < n)
            tokens[tid] = __ldcg(p.tokens + lo + tid);
    }
    __syncthreads();
    if (c >= p.N)
        return;
    float acc[8] = {};
    int run = ids[1];
    bool before = ids[0] == run;  // the run began in an earlier chunk
    auto flush = [&](bool behind) {
        if (!before && !behind) {
            finish_row<W, WIDE>(dtable + run * p.ldt, c, p.N, acc, p.scale, p.accumulate);
        } else {
            float *part = p.parts + (2 * chunk + (before ? 0 : 1)) * p.ld_parts;
            store8<float, WIDE>(part, c, kSumThreads, p.N, acc);
        }
    };
    for (int j0 = 0; j0 < n; j0 += 4) {
        float v[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            load8<D, WIDE>(dd + (j0 + u < n ? tokens[j0 + u] : 0) * p.lddd, c, kSumThreads, j0 + u < n ? p.N : 0, v[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (j0 + u < n) {
                const int id = ids[1 + j0 + u];
                if (id != run) {
                    flush(false);
                    run = id;
                    before = false;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        acc[i] = v[u][i];
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        acc[i] += v[u][i];
                }
            }
        }
    }
    flush(n == p.chunk && ids[p.chunk + 1] == run);
}

// Joins the parts of each run that passes a chunk's end, in the order of the
// chunks: a block for the chunk in which the run begins, its groups of threads
// for equal shares of the chunks behind it.
template <typename W, bool WIDE>
__global__ void __launch_bounds__(kSumThreads * kJoinGroups) embed_join_kernel(W *dtable, const SumParams p)
{
    __shared__ float part[kJoinGroups - 1][8][kSumThreads];
    const int tid = threadIdx.x, group = threadIdx.y;
    const long long chunk = blockIdx.x / p.col_blocks;
    const int c = static_cast<int>(blockIdx.x - chunk * p.col_blocks) * kSumColumns + (WIDE ? 8 : 1) * tid;
    grid_start();
    const long long kept = __ldcg(p.kept), next = (chunk + 1) * p.chunk;
    if (next >= kept)
        return;
    const int run = __ldcg(p.ids + next);
    if (__ldcg(p.ids + next - 1) != run || (chunk > 0 && __ldcg(p.ids + next - p.chunk - 1) == run))
        return;  // no run that begins in this chunk passes its end
    // chunks behind this one that begin with the run: each warp narrows them
    // down to a 32nd at a time
    long long more = 0, most = (kept - next + p.chunk - 1) / p.chunk;  // the first `more` do, those from `most` on do not
    while (more < most) {
        const long long step = (most - more + 31) / 32, i = more + (tid & 31) * step;
        const unsigned yes = __ballot_sync(0xffffffffu, i < most && __ldcg(p.ids + next + min(i, most - 1) * p.chunk) == run);
        const int hits = __popc(yes);  // of ascending i: the first ones
        most = min(most, more + hits * step);
        if (hits > 0)
            more += (hits - 1) * step + 1;
    }
    const long long share = (more + kJoinGroups - 1) / kJoinGroups;
    const long long first = chunk + 1 + group * share, end = min(first + share, chunk + 1 + more);
    float acc[8] = {};
    if (group == 0)
        load8<float, WIDE>(p.parts + (2 * chunk + 1) * p.ld_parts, c, kSumThreads, p.N, acc);
    for (long long k = first; k < end; k += 4) {
        float v[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            load8<float, WIDE>(p.parts + 2 * min(k + u, end - 1) * p.ld_parts, c, kSumThreads, k + u < end ? p.N : 0, v[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[i] += v[u][i];
    }
    if (group > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            part[group - 1][i][tid] = acc[i];
    }
    __syncthreads();
    if (group > 0 || c >= p.N)
        return;
#pragma unroll
    for (int g = 0; g < kJoinGroups - 1; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[i] += part[g][i][tid];
    finish_row<W, WIDE>(dtable + run * p.ldt, c, p.N, acc, p.scale, p.accumulate);
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
    size_t kept, counts, ids_a, tokens_a, ids_b, tokens_b, parts, bytes;  // offsets
    int64_t ld_parts;
};

EmbedPlan embed_plan(int64_t T, int64_t N, int64_t V)
{
    EmbedPlan e = {};
    e.sort = sort_plan(T, V);
    // as long as they leave the SMs four blocks each
    const int64_t col_blocks = (N + kSumColumns - 1) / kSumColumns;
    e.chunk = T * col_blocks >= 32 * kSumBlocks ? 32 : T * col_blocks >= 16 * kSumBlocks ? 16 : 8;
    e.chunks = (T + e.chunk - 1) / e.chunk;
    e.ld_parts = (N + 7) / 8 * 8;
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t o = at;
        at += static_cast<size_t>((bytes + 255) / 256 * 256);
        return o;
    };
    e.kept = take(4);
    e.counts = take(e.sort.blocks > 1 ? static_cast<int64_t>(e.sort.blocks) * 4 << e.sort.bits : 0);
    e.ids_a = take(4 * T);
    e.tokens_a = take(4 * T);
    const bool again = e.sort.passes > 1 && e.sort.blocks > 1;  // one block passes them on through shared memory
    e.ids_b = take(again ? 4 * T : 0);
    e.tokens_b = take(again ? 4 * T : 0);
    e.parts = take(e.chunks > 1 ? 2 * e.chunks * e.ld_parts * 4 : 0);
    e.bytes = at;
    return e;
}

constexpr int kZeroBlocks = 304;  // of 512 threads, beside the sort's; half as many of 1024, of which an SM holds one

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
    const int64_t beside = p.blocks == 1 ? kZeroBlocks / 2 - 1 : kZeroBlocks;
    const unsigned grid = static_cast<unsigned>(p.blocks + (zeros > 0 ? std::min(beside, (zeros + 511) / 512) : 0));
    const size_t smem = static_cast<size_t>(kSortWarps + 2) * p.bins * sizeof(int);
    if (p.blocks == 1) {
        const int most = kBlockWarps * kSortMaxBins * 4 + kBlockMost * 6;
        if (ensure_smem_attribute(sort_block_kernel, most, sort_attribute_set) != cudaSuccess)
            return GEMM_ERR_CUDA;
        return host_launch(sort_block_kernel, grid, 32 * kBlockWarps, static_cast<size_t>(kBlockWarps) * p.bins * 4 + static_cast<size_t>(T) * 6, st,
                           0, p, e.sort.passes, at[0], at[1]);
    }
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
    const int64_t items = wide ? N * type_bytes(d_type) / 16 : N, all = T * items, block = kEmbedThreads * kEmbedItems;
    const int64_t blocks = (all + block - 1) / block;
    if (blocks > kSizeLimit)
        return GEMM_ERR_UNSUPPORTED;
    const bool narrow = blocks * block <= UINT32_MAX;  // items are counted in 32 bits
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return with_type(t_type, [&](auto ttag) {
        using S = decltype(ttag);
        return with_type(d_type, [&](auto dtag) {
            using D_ = decltype(dtag);
            const S *from = static_cast<const S *>(table);
            D_ *to = static_cast<D_ *>(D);
            const unsigned grid = static_cast<unsigned>(blocks), row = static_cast<unsigned>(items);
            const int v = static_cast<int>(V);
            if (narrow)
                return host_launch(wide ? embed_kernel<S, D_, true, unsigned> : embed_kernel<S, D_, false, unsigned>, grid, kEmbedThreads, 0, st, 0,
                                   from, ldt, ids, to, ldd, row, all, v, scale);
            return host_launch(wide ? embed_kernel<S, D_, true, unsigned long long> : embed_kernel<S, D_, false, unsigned long long>, grid,
                               kEmbedThreads, 0, st, 0, from, ldt, ids, to, ldd, row, all, v, scale);
        });
    });
}

size_t gemm_embed_backward_workspace_size(int64_t T, int64_t N, int64_t V)
{
    if (T < 1 || N < 1 || V < 1 || !countable(T) || !countable(N) || !countable(V))
        return 0;
    return embed_plan(T, N, V).bytes;
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
    const size_t need = gemm_embed_backward_workspace_size(T, N, V);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return GEMM_ERR_INVALID_ARG;
    if (need > 0 && !aligned_to(workspace, 256))
        return GEMM_ERR_ALIGNMENT;
    const int64_t col_blocks = (N + kSumColumns - 1) / kSumColumns;
    const EmbedPlan e = embed_plan(std::max<int64_t>(T, 1), N, V);
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
    if ((s = launch_sort(e, sort, T, V, ids, ws, st)) != GEMM_OK)
        return s;
    SumParams p = {};
    p.ids = reinterpret_cast<int *>(ws + e.ids_a);
    p.tokens = reinterpret_cast<int *>(ws + e.tokens_a);
    p.kept = reinterpret_cast<int *>(ws + e.kept);
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
            gemm_status_t r = host_launch(wide ? embed_sum_kernel<D, W, true> : embed_sum_kernel<D, W, false>, grid, kSumThreads, 0, st, 0, from, to, p);
            if (r != GEMM_OK || e.chunks == 1)
                return r;
            return host_launch(wide ? embed_join_kernel<W, true> : embed_join_kernel<W, false>, grid, dim3(kSumThreads, kJoinGroups), 0, st, 0,
                               to, p);
        });
    });
}

}  // extern "C"
