// Expert-layer operators around the products: routing and its gradient, the
// order of the rows by expert, the quantisation of rows to 8 bits, and the
// weighted sum of the experts' rows with its gradient. Contracts are in
// include/gemm_gb300.h.
//
// They read their inputs once, but for the chosen logits of a routing with a
// bias, the ids of an order in several parts (counted, then handed out) and rows
// too long for a block's registers in the quantisation. Sums and softmax
// statistics are fp32 and results are rounded once, on the store. Times in the comments are of one
// launch among others on a GB300 with operands that are not in L2; the HBM
// rate they are set against is 6.78 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/gemm_gb300.h"
#include "host.h"

using namespace g300;

namespace {

// ---------------------------------------------------------------- element access

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x)
{
    return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x)
{
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float x)
{
    return __float2half_rn(x);
}

// Eight elements of a row of n: neighbours from `at`, by 16-byte accesses, when
// WIDE (the address is a multiple of 16 bytes and n one of eight elements),
// else single ones `step` apart, so that the threads lie side by side. Loads
// past the end give zeros.
template <typename T, bool WIDE>
__device__ __forceinline__ void load8(const T *p, int at, int step, int n, float (&v)[8])
{
    if constexpr (WIDE) {
        union {
            uint4 w[sizeof(T) / 2];
            T e[8];
        } u;
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
            u.w[i] = at < n ? reinterpret_cast<const uint4 *>(p + at)[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = to_float(u.e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = at + i * step < n ? to_float(p[at + i * step]) : 0.0f;
    }
}

template <typename T, bool WIDE>
__device__ __forceinline__ void store8(T *p, int at, int step, int n, const float (&v)[8])
{
    if constexpr (WIDE) {
        union {
            uint4 w[sizeof(T) / 2];
            T e[8];
        } u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u.e[i] = from_float<T>(v[i]);
        if (at < n) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
                reinterpret_cast<uint4 *>(p + at)[i] = u.w[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at + i * step < n)
                p[at + i * step] = from_float<T>(v[i]);
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(1.0f + expf(-x)); }

// ---------------------------------------------------------------- routing

// The sigmoid as a choice compares it: to fp32 rounding down to the smallest
// subnormal number, where 1 / (1 + e^-x) would be 0 from x = -88.7 on.
__device__ __forceinline__ float choice_sigmoid(float x)
{
    const float e = expf(-fabsf(x)), r = __frcp_rn(1.0f + e);
    return x < 0.0f ? e * r : r;
}

struct RouteParams {
    long long T;
    int E, k;
    long long ldl;
    const float *bias;
    float *weights;
    int *ids;
    int sigmoid, groups, per, group_top, groups_kept, renorm;
    float scale;
    unsigned int per_inv;  // ceil(2^32 / per): e / per = umulhi(e, per_inv) for per >= 2
    int group_lanes;       // lanes that look through one group
};

// Order-preserving code of a choice value; 0 for what is never chosen (-inf
// and NaN). +0 and -0 get one code.
__device__ __forceinline__ uint32_t choice_key(float v)
{
    if (!(v > -INFINITY))
        return 0u;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

constexpr int kRouteWarps = 4;

// The value a code stands for.
__device__ __forceinline__ float choice_value(uint32_t key)
{
    return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// A lane's two best codes among those not taken.
struct LaneBest {
    uint32_t key, next;
    int i, next_i;
};

template <int NPL>
__device__ __forceinline__ LaneBest lane_best(const uint32_t (&key)[NPL], uint32_t taken)
{
    LaneBest b{0u, 0u, 0, 0};
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const uint32_t v = (taken >> i) & 1u ? 0u : key[i];
        if (v > b.key) {
            b.next = b.key;
            b.next_i = b.i;
            b.key = v;
            b.i = i;
        } else if (v > b.next) {
            b.next = v;
            b.next_i = i;
        }
    }
    return b;
}

// One warp per token; lane l holds experts l, l + 32, ... (NPL of them). The
// k best are taken one at a time: a warp-wide integer maximum of the lanes'
// best codes, then the lowest expert among the lanes that hold it. A lane keeps
// its two best, so it looks through its codes again only when both are taken.
//
// s = softmax(l) or sigmoid(l); e is chosen by s_e + bias_e; w = s / sum of the
// chosen s. Both the compared scores and the weights are fp32, by expf. For
// 16384 tokens memory could deliver in 0.4 (64 experts, bf16) to 2.6 us (256,
// fp32); the kernel takes 8.2 us (k = 6, no bias; 467 instructions a token) and
// 17.4 us (k = 8 with a bias, 1003; 24.2 us with 8 groups): held by the instructions
// it issues, of which the k rounds of maxima across the warp are most. Before the
// lanes kept two candidates the second took 25 us. Special-function scores took
// 14.6 and 21.5 us, but flushed those below 2^-126 and tied their experts. One
// token takes 2.4 us, launch latency.
template <typename L, int NPL>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const L *logits, const RouteParams p)
{
    extern __shared__ float group_smem[];  // per warp: groups x (per | 1) choice values
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + warp;
    grid_start();
    if (t >= p.T)
        return;
    const L *row = logits + t * p.ldl;
    float l[NPL];
    float top = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < p.E ? to_float(row[e]) : -INFINITY;
    }
    float bias[NPL];  // asked for with the logits: one wait for memory
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            bias[i] = lane + 32 * i < p.E ? p.bias[lane + 32 * i] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        bad |= l[i] != l[i] || (!p.sigmoid && l[i] == INFINITY);
        top = fmaxf(top, l[i]);
    }
    bad = __any_sync(0xffffffffu, bad);
    // the softmax over all experts: needed for the weights when they are not
    // renormalised (renormalised ones are a softmax over the chosen), and for
    // the choice when a bias is added to the scores or groups are summed
    const bool scored = p.bias || p.groups > 1;
    float s[NPL];
    float total = 1.0f;
    if (!p.sigmoid) {
        top = warp_max(top);
        if (top == -INFINITY)
            top = 0.0f;
        if (!p.renorm || scored) {
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                // a logit of +inf counts as 1 beside others of 0, so that the choice has its order
                s[i] = l[i] == top ? 1.0f : l[i] > -INFINITY ? expf(l[i] - top) : 0.0f;
                total += s[i];
            }
            total = warp_sum(total);
            if (total == 0.0f)
                total = 1.0f;
        }
    }
    // what the choice goes by
    uint32_t key[NPL];
    if (scored) {
        const float inv = __frcp_rn(total);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            s[i] = p.sigmoid ? choice_sigmoid(l[i]) : s[i] * inv;
            if (p.bias)
                s[i] = __fadd_rn(s[i], bias[i]);
            key[i] = l[i] > -INFINITY ? choice_key(p.bias ? s[i] : l[i]) : 0u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            key[i] = choice_key(l[i]);
    }
    if (p.groups > 1) {
        const int stride = p.per | 1;  // odd: lanes reading one value of each group meet distinct banks
        float *gs = group_smem + warp * p.groups * stride;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 32 * i;
            if (e < p.E) {
                const int g = p.per == 1 ? e : static_cast<int>(__umulhi(static_cast<unsigned>(e), p.per_inv));
                gs[g * stride + e - g * p.per] = key[i] != 0u ? s[i] : -INFINITY;
            }
        }
        __syncwarp();
        // the two best of each group, by 32 / groups (rounded down to a power of two) lanes
        const int sub = p.group_lanes, g_of = lane / sub;
        float a = -INFINITY, b = -INFINITY;
        if (g_of < p.groups) {
#pragma unroll 4
            for (int i = lane % sub; i < p.per; i += sub) {
                const float v = gs[g_of * stride + i];
                b = fmaxf(b, fminf(a, v));
                a = fmaxf(a, v);
            }
        }
        for (int o = 1; o < sub; o <<= 1) {
            const float oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
            b = fmaxf(fminf(a, oa), fmaxf(b, ob));
            a = fmaxf(a, oa);
        }
        // lane g takes group g's score
        uint32_t gkey = 0u;
        if (a > -INFINITY)
            gkey = choice_key(p.group_top == 2 && b > -INFINITY ? __fadd_rn(a, b) : a);
        gkey = __shfl_sync(0xffffffffu, gkey, (lane * sub) & 31);
        if (lane >= p.groups)
            gkey = 0u;
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const uint32_t o = __shfl_sync(0xffffffffu, gkey, g);
            rank += o > gkey || (o == gkey && g < lane);
        }
        const uint32_t kept = __ballot_sync(0xffffffffu, gkey != 0u && rank < p.groups_kept);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 32 * i;
            if (e < p.E) {
                const int g = p.per == 1 ? e : static_cast<int>(__umulhi(static_cast<unsigned>(e), p.per_inv));
                if (!((kept >> g) & 1u))
                    key[i] = 0u;
            }
        }
    }
    // the k best; lane j keeps the j-th
    int my_id = -1;
    uint32_t my_key = 0u, taken = 0u;
    LaneBest best = lane_best<NPL>(key, 0u);
    bool fresh = true;  // best.next is known
    for (int j = 0; j < p.k; ++j) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, best.key);
        if (m == 0u)
            break;
        const uint32_t who = __ballot_sync(0xffffffffu, best.key == m);
        int e = lane + 32 * best.i;
        if (who & (who - 1))  // lanes that tie: the lowest expert
            e = static_cast<int>(__reduce_min_sync(0xffffffffu, static_cast<unsigned>(best.key == m ? e : INT_MAX)));
        else
            e = __shfl_sync(0xffffffffu, e, __ffs(who) - 1);
        if (lane == j) {
            my_id = e;
            my_key = m;
        }
        if (lane == (e & 31)) {
            taken |= 1u << best.i;
            if (fresh) {
                best.key = best.next;
                best.i = best.next_i;
            } else {
                best = lane_best<NPL>(key, taken);
            }
            fresh = !fresh;
        }
    }
    // weights of the chosen, one lane each
    const float my_l = my_id < 0 ? -INFINITY : p.bias ? to_float(row[my_id]) : choice_value(my_key);
    float w = 0.0f;
    if (p.sigmoid) {
        if (my_id >= 0)
            w = sigmoid(my_l);
    } else if (p.renorm) {
        const float m = warp_max(my_l);  // relative to the largest chosen logit: its term is 1, the sum never 0
        if (my_id >= 0)
            w = expf(my_l - m);
    } else if (my_id >= 0) {
        w = __fdiv_rn(expf(my_l - top), total);
    }
    if (p.renorm) {
        const float sum = warp_sum(w);
        w = __fdiv_rn(w, sum == 0.0f ? 1.0f : sum);
    }
    if (lane < p.k) {
        p.weights[t * p.k + lane] = bad ? NAN : w * p.scale;
        p.ids[t * p.k + lane] = my_id;
    }
}

struct RouteGradParams {
    long long T;
    int E, k;
    long long ldl, lddl;
    const int *ids;
    const float *dweights;
    int sigmoid, renorm;
    float scale;
};

// One warp per token. The chosen experts' values are computed one lane each
// and put into a shared-memory row of zeros, which is then written whole;
// only the softmax over all experts (FULL) reads the other logits, which it
// holds in registers (NPL a lane) from the maximum to the gradient.
//
// sigmoid: dl = ds s (1 - s); softmax: dl = s (ds - sum ds s); renormalised
// weights w = s / P: ds = (g - sum g w) / P over the chosen. Bound by the
// writing of dlogits, 2.5 us for 16384 x 256 fp32: 7.4 us for sigmoid scores;
// 9.9 us with the softmax over all (12.5 when the logits were read three times).
template <typename L, int NPL, bool FULL>
__global__ void __launch_bounds__(32 * kRouteWarps)
    route_backward_kernel(const L *logits, L *__restrict__ dlogits, const RouteGradParams p)
{
    extern __shared__ float grad_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + warp;
    float *ds = grad_smem + warp * p.E;
    if (t < p.T)
        for (int e = lane; e < p.E; e += 32)
            ds[e] = 0.0f;
    grid_start();
    if (t >= p.T)
        return;
    const L *row = logits + t * p.ldl;
    L *out = dlogits + t * p.lddl;
    int id = -1;
    float g = 0.0f, x = -INFINITY;
    float s[NPL];
    if constexpr (FULL) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 32 * i;
            s[i] = e < p.E ? to_float(row[e]) : -INFINITY;
        }
    }
    if (lane < p.k) {
        id = p.ids[t * p.k + lane];
        if (id < 0 || id >= p.E)
            id = -1;
        if (id >= 0) {
            g = p.dweights[t * p.k + lane] * p.scale;
            x = to_float(row[id]);
        }
    }
    __syncwarp();
    if constexpr (FULL) {
        // dl_e = s_e (ds_e - sum ds s)
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            top = fmaxf(top, s[i]);
        top = warp_max(top);
        if (top == -INFINITY)
            top = 0.0f;
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            s[i] = expf(s[i] - top);
            total += s[i];
        }
        total = warp_sum(total);
        if (total == 0.0f)
            total = 1.0f;
        const float dot = warp_sum(id >= 0 ? g * __fdiv_rn(expf(x - top), total) : 0.0f);
        if (id >= 0)
            ds[id] = g;
        __syncwarp();
        const float inv = __frcp_rn(total);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 32 * i;
            if (e < p.E)
                out[e] = from_float<L>(s[i] * inv * (ds[e] - dot));
        }
    } else {
        // share of the chosen score in the sum, and d score / d logit over the score
        float c = 0.0f, rest = 1.0f;
        if (p.sigmoid) {
            if (id >= 0) {
                c = sigmoid(x);
                rest = sigmoid(-x);  // 1 - s without its cancellation
            }
        } else {
            const float m = warp_max(x);
            if (id >= 0)
                c = expf(x - m);
        }
        float d = g * c * rest;
        if (p.renorm) {
            float sum = warp_sum(c);
            if (sum == 0.0f)
                sum = 1.0f;
            const float w = __fdiv_rn(c, sum);
            d = w * (g - warp_sum(g * w)) * rest;
        }
        if (id >= 0)
            ds[id] = d;
        __syncwarp();
#pragma unroll 8
        for (int e = lane; e < p.E; e += 32)
            out[e] = from_float<L>(ds[e]);
    }
}

// ---------------------------------------------------------------- order by expert
//
// A stable counting sort. The pairs are cut into one contiguous part per
// block, a part into one run per warp. plan_count_kernel leaves each part's
// count of every expert; plan_scatter_kernel adds the counts of the parts and
// warps before it and hands out the rows in order, 32 pairs at a time. One
// part needs no count kernel. Bound by latency: a chain of counting, a scan and
// the hand-out, 2.3 us for one token's pairs, 8.0 us for the 131072 of 16384
// tokens (0.2 us of traffic); the parts' counts were 14 us when each thread
// added up all parts of its expert.

constexpr int kPlanMaxWarps = 16;
constexpr int kPlanPart = 2048;      // pairs per block before more blocks are taken
constexpr int kPlanMaxBlocks = 128;  // every block reads the counts of all: more cost more than they give

// Warps per block: about four steps of 32 pairs for each, and few enough that
// their counts of all experts share 48 KB of memory.
inline int plan_warps(int64_t part, int64_t E)
{
    const int most = E <= 512 ? kPlanMaxWarps : kPlanMaxWarps / 2;
    return part <= 512 ? 4 : part <= 1024 ? 8 : most;
}

__host__ __device__ inline int plan_blocks(long long pairs)
{
    const long long b = (pairs + kPlanPart - 1) / kPlanPart;
    return static_cast<int>(b < 1 ? 1 : b > kPlanMaxBlocks ? kPlanMaxBlocks : b);
}

constexpr int kPlanBatch = 4;  // ids a lane loads at a time

// The ids of pairs i, i + 32, ... below `end`; -1 for those outside 0..E-1.
// Through L2: plan_scatter_kernel reads them before its own grid_start().
__device__ __forceinline__ void plan_load(const int *ids, long long i, long long end, int E, int (&id)[kPlanBatch])
{
#pragma unroll
    for (int u = 0; u < kPlanBatch; ++u)
        id[u] = i + 32 * u < end ? __ldcg(ids + i + 32 * u) : -1;
#pragma unroll
    for (int u = 0; u < kPlanBatch; ++u)
        if (id[u] < 0 || id[u] >= E)
            id[u] = -1;
}

__global__ void __launch_bounds__(32 * kPlanMaxWarps)
    plan_count_kernel(const int *ids, long long pairs, long long part, int E, int *counts)
{
    extern __shared__ int plan_smem[];
    // the ids are written; only then may plan_scatter_kernel start, which
    // counts them for itself before it waits for this kernel
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        plan_smem[e] = 0;
    __syncthreads();
    const long long lo = blockIdx.x * part, hi = min(lo + part, pairs);
    const int warp = threadIdx.x >> 5, warps = static_cast<int>(blockDim.x >> 5), lane = threadIdx.x & 31;
    for (long long i0 = lo + 32 * kPlanBatch * warp; i0 < hi; i0 += 32 * kPlanBatch * warps) {
        int id[kPlanBatch];
        plan_load(ids, i0 + lane, hi, E, id);
#pragma unroll
        for (int u = 0; u < kPlanBatch; ++u)
            if (id[u] >= 0)
                atomicAdd(&plan_smem[id[u]], 1);  // a count: the order of the additions does not show
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        counts[static_cast<long long>(blockIdx.x) * E + e] = plan_smem[e];
}

// Shared memory: warps x E counts, E totals, E rows of the parts before.
__global__ void __launch_bounds__(32 * kPlanMaxWarps)
    plan_scatter_kernel(const int *ids, long long pairs, long long part, int E, int k,
                        const int *counts, int *offsets, int *slots,
                        int *tokens)
{
    extern __shared__ int plan_smem[];
    int *hist = plan_smem;                  // [warp][E]
    const int warps = static_cast<int>(blockDim.x >> 5);
    int *start = plan_smem + warps * E;  // first row of each expert
    int *before = start + E;
    __shared__ int warp_total[kPlanMaxWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long lo = blockIdx.x * part, hi = min(lo + part, pairs);
    const long long run = (((hi > lo ? hi - lo : 0) + warps - 1) / warps + 31) / 32 * 32;
    const long long wlo = min(lo + warp * run, hi), whi = min(wlo + run, hi);
    if (gridDim.x == 1)
        grid_start();
    for (int i = tid; i < (warps + 2) * E; i += blockDim.x)
        hist[i] = 0;
    __syncthreads();
    int first[kPlanBatch];  // the warp's first pairs (mostly all of them) are kept for the hand-out
    plan_load(ids, wlo + lane, whi, E, first);
    for (long long i0 = wlo; i0 < whi; i0 += 32 * kPlanBatch) {
        int id[kPlanBatch];
        if (i0 > wlo)
            plan_load(ids, i0 + lane, whi, E, id);
#pragma unroll
        for (int u = 0; u < kPlanBatch; ++u) {
            const int e = i0 > wlo ? id[u] : first[u];
            if (e >= 0)
                atomicAdd(&hist[warp * E + e], 1);
        }
    }
    __syncthreads();
    // totals of every expert, and of the parts before this one: with several
    // parts all threads add up the counts, `lanes` of them for each expert
    if (gridDim.x == 1) {
        for (int e = tid; e < E; e += blockDim.x) {
            int total = 0;
            for (int w = 0; w < warps; ++w)
                total += hist[w * E + e];
            start[e] = total;
        }
    } else {
        grid_start();  // the counts of all parts are written
        const int lanes = max(1, static_cast<int>(blockDim.x) / E);
        for (int i = tid; i < E * lanes; i += blockDim.x) {
            const int e = i % E;
            int total = 0, prior = 0;
#pragma unroll 16
            for (int b = i / E; b < static_cast<int>(gridDim.x); b += lanes) {
                const int c = __ldcg(counts + static_cast<long long>(b) * E + e);
                total += c;
                prior += b < static_cast<int>(blockIdx.x) ? c : 0;
            }
            atomicAdd(&start[e], total);  // whole numbers: the order of the additions does not show
            atomicAdd(&before[e], prior);
        }
    }
    __syncthreads();
    // exclusive scan of the totals: each warp takes a run of experts, one lane
    // a part of it
    const int per = (E + 32 * warps - 1) / (32 * warps);
    const int e0 = min(tid * per, E), e1 = min(e0 + per, E);
    int sum = 0;
    for (int e = e0; e < e1; ++e)
        sum += start[e];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        warp_total[warp] = incl;
    __syncthreads();
    int base = incl - sum, kept = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp)
            base += warp_total[w];
        kept += warp_total[w];
    }
    for (int e = e0; e < e1; ++e) {
        const int n = start[e];
        start[e] = base;
        base += n;
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int e = tid; e < E; e += blockDim.x)
            offsets[e] = start[e];
        if (tid == 0)
            offsets[E] = kept;
    }
    // first row of each warp's pairs of each expert
    for (int e = tid; e < E; e += blockDim.x) {
        int at = start[e] + before[e];
        int n[kPlanMaxWarps];
#pragma unroll
        for (int w = 0; w < kPlanMaxWarps; ++w)
            n[w] = w < warps ? hist[w * E + e] : 0;
#pragma unroll
        for (int w = 0; w < kPlanMaxWarps; ++w) {
            if (w < warps)
                hist[w * E + e] = at;
            at += n[w];
        }
    }
    __syncthreads();
    int *mine = hist + warp * E;
    for (long long i0 = wlo; i0 < whi; i0 += 32 * kPlanBatch) {
        int id[kPlanBatch];
        if (i0 > wlo)
            plan_load(ids, i0 + lane, whi, E, id);
#pragma unroll
        for (int u = 0; u < kPlanBatch; ++u) {
            const long long i = i0 + 32 * u + lane;
            const int e = i0 > wlo ? id[u] : first[u];
            const unsigned same = __match_any_sync(0xffffffffu, e);
            int slot = -1;
            if (e >= 0)
                slot = mine[e] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (e >= 0 && (same >> lane) == 1u)  // the last of its expert moves the count on
                mine[e] = slot + 1;
            __syncwarp();
            if (i < whi) {
                slots[i] = slot;
                if (slot >= 0)
                    tokens[slot] = static_cast<int>(static_cast<unsigned>(i) / static_cast<unsigned>(k));
            }
        }
    }
    // rows that no pair has
    for (long long i = kept + static_cast<long long>(blockIdx.x) * blockDim.x + tid; i < pairs;
         i += static_cast<long long>(gridDim.x) * blockDim.x)
        tokens[i] = -1;
}

// ---------------------------------------------------------------- quantisation

struct QuantParams {
    long long M;
    int K;
    const int *index;
    long long x_rows, ldx, ldq;
    float *scales;
};

constexpr int kQuantMaxThreads = 512;
constexpr int kQuantShared = 256;  // threads of a block of several rows
constexpr int kQuantMany = 1024;   // rows

// Eight elements of one type, in registers.
template <typename T>
struct Eight {
    union {
        uint4 w[sizeof(T) / 2];
        T e[8];
    };
    __device__ __forceinline__ Eight() {}
};

// A row's elements at .. at+7 from 16-byte words, its address and `at` a
// multiple of 16 bytes and of 8; zeros unless `in`.
template <typename T>
__device__ __forceinline__ void load_wide(const T *row, int at, bool in, Eight<T> &v)
{
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
        v.w[i] = in ? reinterpret_cast<const uint4 *>(row + at)[i] : make_uint4(0, 0, 0, 0);
}

// Whether the whole 16-byte words around elements at .. at+7 lie inside a row of n, whatever its address.
template <typename T>
__device__ __forceinline__ bool inside(int at, int n)
{
    constexpr int word = 16 / sizeof(T);
    return at >= word && at <= n - 8 - word;
}

// The same elements at any address, from the aligned words around them, which
// are shifted into place (a neighbour's second word is the next thread's
// first, in L1): 1000 rows of 8191 bf16 in 9.9 us, 24.4 by single elements.
// Zeros unless `in`.
template <typename T>
__device__ __forceinline__ void load_shifted(const T *row, int at, bool in, Eight<T> &v)
{
    constexpr int W = sizeof(T) / 2;
    const uintptr_t address = reinterpret_cast<uintptr_t>(row + at);
    const uint4 *from = reinterpret_cast<const uint4 *>(address & ~static_cast<uintptr_t>(15));
    const uint32_t shift = static_cast<uint32_t>(address) & 15u;
    uint32_t r[4 * W + 4];
#pragma unroll
    for (int i = 0; i <= W; ++i) {
        const uint4 x = in ? from[i] : make_uint4(0, 0, 0, 0);
        r[4 * i] = x.x;
        r[4 * i + 1] = x.y;
        r[4 * i + 2] = x.z;
        r[4 * i + 3] = x.w;
    }
#pragma unroll
    for (int i = 0; i < 4 * W + 2; ++i)
        r[i] = shift & 8u ? r[i + 2] : r[i];
#pragma unroll
    for (int i = 0; i < 4 * W + 1; ++i)
        r[i] = shift & 4u ? r[i + 1] : r[i];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        v.w[i].x = __funnelshift_r(r[4 * i], r[4 * i + 1], 8 * (shift & 3u));
        v.w[i].y = __funnelshift_r(r[4 * i + 1], r[4 * i + 2], 8 * (shift & 3u));
        v.w[i].z = __funnelshift_r(r[4 * i + 2], r[4 * i + 3], 8 * (shift & 3u));
        v.w[i].w = __funnelshift_r(r[4 * i + 3], r[4 * i + 4], 8 * (shift & 3u));
    }
}

// The same one by one, zeros past the end: the ends of a row.
template <typename T>
__device__ __forceinline__ void load_single(const T *row, int at, int n, Eight<T> &v)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v.e[i] = at + i < n ? row[at + i] : from_float<T>(0.0f);
}

// A chunk as loaded (PLAIN), so that it takes no more registers than its bytes
// until it is rounded, or gated.
template <typename X, bool GATED>
struct QuantChunk : Eight<typename std::conditional<GATED, float, X>::type> {
    using Store = typename std::conditional<GATED, float, X>::type;
    __device__ __forceinline__ float at(int i) const { return to_float(this->e[i]); }
};

// Columns past K, and rows that do not exist (K 0), are zeros. A PLAIN chunk at
// the end of a row that is not WIDE is left to quant_end, so that nothing stands
// between the loads of one chunk and the next.
template <typename X, bool GATED, bool WIDE>
__device__ __forceinline__ void quant_load(const X *row, int at, int K, QuantChunk<X, GATED> &v)
{
    if constexpr (GATED) {
        Eight<X> g, u;
        if constexpr (WIDE) {
            load_wide(row, at, at < K, g);
            load_wide(row + K, at, at < K, u);
        } else if (inside<X>(at, K)) {
            load_shifted(row, at, true, g);
            load_shifted(row + K, at, true, u);
        } else {
            load_single(row, at, K, g);
            load_single(row + K, at, K, u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // silu(gate) * up
            const float x = to_float(g.e[i]);
            v.e[i] = __fmul_rn(__fdiv_rn(x, 1.0f + expf(-x)), to_float(u.e[i]));
        }
    } else if constexpr (WIDE) {
        load_wide(row, at, at < K, v);
    } else {
        load_shifted(row, at, inside<X>(at, K), v);
    }
}

template <typename X, bool GATED, bool WIDE>
__device__ __forceinline__ void quant_end(const X *row, int at, int K, QuantChunk<X, GATED> &v)
{
    if constexpr (!GATED && !WIDE) {
        if (at < K && !inside<X>(at, K))
            load_single(row, at, K, v);
    }
}

// The largest magnitude of a chunk and `top`, as the bits of a nonnegative
// fp32 number, whose order as integers puts infinities and NaN last.
template <typename X, bool GATED>
__device__ __forceinline__ uint32_t quant_top(const QuantChunk<X, GATED> &v, uint32_t top)
{
    if constexpr (sizeof(typename QuantChunk<X, GATED>::Store) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            top = max(top, __float_as_uint(v.e[i]) & 0x7fffffffu);
    } else {
        // sixteen-bit codes without their signs have the same order
        const uint32_t *w = reinterpret_cast<const uint32_t *>(v.w);
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
        X e;
        *reinterpret_cast<unsigned short *>(&e) = static_cast<unsigned short>(m);
        top = max(top, __float_as_uint(to_float(e)) & 0x7fffffffu);
    }
    return top;
}

// Two fp32 numbers in a register pair, and a * b + c of each.
__device__ __forceinline__ uint64_t pair_of(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ void pair_to(uint64_t p, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}

// round(x / scale) to whole numbers of at most 127, exactly that of the
// correctly rounded quotient: x times the reciprocal is within 3e-5 of it, so
// only where that lies near a half is the quotient itself taken. Adding
// 1.5 * 2^23 rounds to a whole number and leaves it in the low byte.
__device__ __forceinline__ void quant_round(const float (&x)[8], float scale, float inv, bool exact, uint32_t (&q)[8])
{
    const uint64_t magic = pair_of(12582912.0f, 12582912.0f), minus = pair_of(-1.0f, -1.0f), inv2 = pair_of(inv, inv);
    float near_half = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint64_t two = pair_of(x[i], x[i + 1]);
        const uint64_t t = fma_pair(two, inv2, magic);
        const uint64_t off = fma_pair(two, inv2, fma_pair(t, minus, magic));  // x / scale less the whole number
        float a, b;
        pair_to(off, a, b);
        near_half = fmaxf(near_half, fmaxf(fabsf(a), fabsf(b)));
        pair_to(t, a, b);
        q[i] = __float_as_uint(a);
        q[i + 1] = __float_as_uint(b);
    }
    if (exact || near_half > 0.4999f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q[i] = static_cast<uint32_t>(max(-127, min(127, __float2int_rn(__fdiv_rn(x[i], scale)))));
    }
}

// The block's x threads take a row, several rows a block (y) where they are
// short; CH chunks of 8 elements a thread kept in registers between the maximum
// and the rounding (CH 0: rows too long for that are read twice, the second
// time from L2). WIDE: rows of 16-byte words. Bound by memory, and by the pause
// between a row's loads and its stores, which three blocks an SM cover in part:
// 8192 x 8192 bf16 in 42.3 us (4.8 TB/s; 64 with a division for each element,
// 47 with two blocks an SM, 44.2 without the paired arithmetic of quant_round;
// a kernel that issues instructions three cycles of four), 1536 gated rows of 2048 from fp32 in 7.2 us, rows
// of odd length (4096 x 4001) in 17 us; four chunks a thread of those want the
// registers of two blocks an SM (1000 x 8191: 11.5 us with three, 9.9 with two).
template <typename X, bool GATED, bool WIDE, int CH>
__global__ void __launch_bounds__(kQuantMaxThreads, WIDE || CH < 4 ? 3 : 2)
    quantize_kernel(const X *x, int8_t *__restrict__ q, const QuantParams p)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = static_cast<int>(blockDim.x >> 5);
    const long long m = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    // a thread's chunk c is the eight columns from at0 + c * step
    const int at0 = 8 * tid, step = 8 * static_cast<int>(blockDim.x);
    __shared__ uint32_t warp_top[kQuantMaxThreads / 32];
    grid_start();
    const bool have = m < p.M;
    const long long r = !have ? -1 : p.index ? p.index[m] : m;
    const bool live = r >= 0 && r < p.x_rows;
    const int K = live ? p.K : 0;
    const X *row = x + (live ? r : 0) * p.ldx;
    const int chunks = CH ? CH : (p.K + step - 1) / step;
    QuantChunk<X, GATED> v[CH ? CH : 1];
    uint32_t top = 0u;
    if constexpr (CH > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            quant_load<X, GATED, WIDE>(row, at0 + c * step, K, v[c]);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            quant_end<X, GATED, WIDE>(row, at0 + c * step, K, v[c]);
            top = quant_top(v[c], top);
        }
    } else {
        for (int c = 0; c < chunks; ++c) {
            quant_load<X, GATED, WIDE>(row, at0 + c * step, K, v[0]);
            quant_end<X, GATED, WIDE>(row, at0 + c * step, K, v[0]);
            top = quant_top(v[0], top);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (warps > 1) {
        uint32_t *tops = warp_top + threadIdx.y * warps;
        if (lane == 0)
            tops[warp] = top;
        __syncthreads();
        top = __reduce_max_sync(0xffffffffu, lane < warps ? tops[lane] : 0u);
    }
    if (!have)
        return;
    const bool bad = top >= 0x7f800000u;  // the row holds an infinity or a NaN
    const float scale = bad ? NAN : __fmul_rn(__uint_as_float(top), 1.0f / 127.0f);
    if (tid == 0)
        p.scales[m] = scale;
    // a scale that is 0 (also: rounded to 0) divides by 1 and leaves zeros; one
    // that is subnormal is divided by, its reciprocal being infinite or its
    // rounding coarse enough for quotients above 127
    const float by = bad || scale == 0.0f ? 1.0f : scale;
    const float inv = __frcp_rn(by);
    const bool exact = by < 1.17549435e-38f;
    int8_t *out = q + m * p.ldq;
    const bool out_wide = (reinterpret_cast<uintptr_t>(out) & 7u) == 0;
    auto write = [&](int c, const QuantChunk<X, GATED> &e) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = e.at(i);
        uint32_t b[8];
        quant_round(f, by, inv, exact, b);
        const int at = at0 + c * step;
        if (WIDE ? at < p.K : out_wide && at <= p.K - 8) {
            const uint32_t lo = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
            const uint32_t hi = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
            *reinterpret_cast<uint2 *>(out + at) = bad ? make_uint2(0u, 0u) : make_uint2(lo, hi);
        } else if constexpr (!WIDE) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (at + i < p.K)
                    out[at + i] = bad ? static_cast<int8_t>(0) : static_cast<int8_t>(b[i] & 0xffu);
        }
    };
    if constexpr (CH > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            write(c, v[c]);
    } else {
        for (int c = 0; c < chunks; ++c) {
            quant_load<X, GATED, WIDE>(row, at0 + c * step, K, v[0]);
            quant_end<X, GATED, WIDE>(row, at0 + c * step, K, v[0]);
            write(c, v[0]);
        }
    }
}

// ---------------------------------------------------------------- weighted sums

struct CombineParams {
    long long T;
    int N, k;
    long long y_rows, ldy, ldd;
    const int *slots;
    const float *weights;
};

constexpr int kCombineThreads = 128;

// D_t = sum_j w_tj Y[slot_tj]: one block per token and 1024 columns; each thread
// sums 8 columns over the k rows. Bound
// by the reading of Y: 4096 tokens, k = 6, N = 4096 bf16 in 41.6 us (0.83 of
// the HBM rate).
template <typename Y, typename D, bool WIDE>
__global__ void __launch_bounds__(kCombineThreads)
    combine_kernel(const Y *y, D *__restrict__ d, const CombineParams p, int col_blocks)
{
    const long long t = blockIdx.x / col_blocks;
    const int c0 = static_cast<int>(blockIdx.x % col_blocks) * (8 * kCombineThreads);
    const int c = c0 + (WIDE ? 8 : 1) * static_cast<int>(threadIdx.x);
    grid_start();
    if (c >= p.N)
        return;
    const int *slots = p.slots + t * p.k;
    const float *weights = p.weights + t * p.k;
    float acc[8] = {};
    // more rows in flight only where loads are narrow: 256 x 2048, k = 6, fp32 in 4.8 us by two, 5.9 by four;
    // 4096 x 4001 bf16 in 57.5 and 53.6
#pragma unroll(WIDE ? 2 : 4)
    for (int j = 0; j < p.k; ++j) {
        const int r = slots[j];
        if (r >= 0 && r < p.y_rows) {
            const float w = weights[j];
            float v[8];
            load8<Y, WIDE>(y + r * p.ldy, c, kCombineThreads, p.N, v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[i] = fmaf(w, v[i], acc[i]);
        }
    }
    store8<D, WIDE>(d + t * p.ldd, c, kCombineThreads, p.N, acc);
}

struct CombineGradParams {
    long long T;
    int N, k;
    long long y_rows, ldy, lddy, lddd;
    const int *slots;
    const float *weights;
    float *dweights;
};

// 256 tokens of 2048, k = 6, fp32: 8.9 us by four warps a block, 9.8 by eight
constexpr int kCombineGradWarps = 4;

// Few pairs of long rows: each has all warps of a block (SHARED), or a warp
// would walk its row alone. us with a warp and with a block a pair: 8 pairs of
// 4096 bf16 5.0, 2.2; 1536 of 2048 bf16 5.4, 3.5, fp32 8.6, 6.6; 4096 of 4096
// fp32 26.9, 25.1; 3332 odd rows of 2005 17.4, 12.0. More, or shorter, lose by it:
// 8192 of 2048 bf16 13.8, 16.4; 4096 of 512 3.3, 4.5, of 1024 5.3, 5.5.
inline bool combine_grad_shared(int64_t pairs, int64_t N) { return N > 256 && pairs <= (N > 1024 ? 4096 : 1024); }

// dY[slot] = w dD, dw = <dD, Y[slot]>: one warp per (token, choice) pair (SHARED:
// the block's warps in turn) walks the N columns once, writing the row of dY and
// summing the dot product; a token's warps share dD's row in L1. Rows that do not
// start on 16-byte words are read by single elements side by side: by the words
// around them, shifted, 24576 odd rows of 4001 bf16 took 127 us instead of 102. Bound by memory: 4096 tokens, k = 6, N =
// 4096 bf16 in 70.1 us (0.92 of the HBM rate).
template <typename Y, typename D, bool WIDE, bool SHARED>
__global__ void __launch_bounds__(32 * kCombineGradWarps)
    combine_backward_kernel(const D *dd, const Y *y, Y *__restrict__ dy,
                            const CombineGradParams p)
{
    const int lane = threadIdx.x & 31, warp = static_cast<int>(threadIdx.x >> 5);
    const long long pair = SHARED ? blockIdx.x : static_cast<long long>(blockIdx.x) * kCombineGradWarps + warp;
    __shared__ float part[kCombineGradWarps];
    grid_start();
    if (pair >= p.T * p.k)
        return;
    const long long t = pair / p.k;
    const int r = p.slots[pair];
    float dot = 0.0f;
    if (r >= 0 && r < p.y_rows) {
        const float w = p.weights[pair];
        const D *g = dd + t * p.lddd;
        const Y *yr = y + r * p.ldy;
        Y *o = dy + r * p.lddy;
#pragma unroll 4
        for (int c0 = SHARED ? 256 * warp : 0; c0 < p.N; c0 += SHARED ? 256 * kCombineGradWarps : 256) {
            const int c = c0 + (WIDE ? 8 : 1) * lane;
            float a[8], b[8];
            load8<D, WIDE>(g, c, 32, p.N, a);
            load8<Y, WIDE>(yr, c, 32, p.N, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dot = fmaf(a[i], b[i], dot);
                b[i] = w * a[i];
            }
            store8<Y, WIDE>(o, c, 32, p.N, b);
        }
    }
    dot = warp_sum(dot);
    if constexpr (SHARED) {
        if (lane == 0)
            part[warp] = dot;
        __syncthreads();
        dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kCombineGradWarps; ++i)
            dot += part[i];
    }
    if (lane == 0 && (!SHARED || warp == 0))
        p.dweights[pair] = dot;
}

// ---------------------------------------------------------------- host

// Calls fn with a value of the element type `type` names.
template <typename F>
gemm_status_t with_type(int type, F fn)
{
    switch (type) {
    case GEMM_OUT_F32: return fn(float());
    case GEMM_OUT_BF16: return fn(__nv_bfloat16());
    case GEMM_OUT_F16: return fn(__half());
    }
    return GEMM_ERR_INVALID_ARG;
}

// The rule of a call with its defaults filled in; false if it makes no sense for E experts and k choices.
bool route_rule(const gemm_route_t *route, int64_t E, int k, gemm_route_t *r)
{
    gemm_route_t d = {};
    *r = route ? *route : d;
    if (r->score != GEMM_ROUTE_SOFTMAX && r->score != GEMM_ROUTE_SIGMOID)
        return false;
    if (r->groups < 0 || r->group_top < 0 || r->group_top > 2 || r->groups_kept < 0 || !std::isfinite(r->scale))
        return false;
    if (r->scale == 0.0f)
        r->scale = 1.0f;
    if (r->groups == 0)
        r->groups = 1;
    if (r->group_top == 0)
        r->group_top = 1;
    if (E < 1 || E > GEMM_ROUTE_MAX_EXPERTS || k < 1 || k > GEMM_ROUTE_MAX_K || k > E)
        return false;
    if (r->groups > 1) {
        if (r->groups > 32 || E % r->groups != 0 || r->groups_kept < 1 || r->groups_kept > r->groups)
            return false;
        const int64_t per = E / r->groups;
        if (r->group_top > per || k > per * r->groups_kept)
            return false;
    }
    return true;
}

template <typename L, int NPL>
gemm_status_t launch_route(const void *logits, const RouteParams &p, cudaStream_t st)
{
    const long long blocks = (p.T + kRouteWarps - 1) / kRouteWarps;
    const size_t smem = p.groups > 1 ? sizeof(float) * kRouteWarps * p.groups * (p.per | 1) : 0;
    return host_launch(route_kernel<L, NPL>, static_cast<unsigned>(blocks), 32 * kRouteWarps, smem, st, 0,
                       static_cast<const L *>(logits), p);
}

template <typename L, int NPL, bool FULL>
gemm_status_t launch_route_backward(const void *logits, void *dlogits, const RouteGradParams &p, cudaStream_t st)
{
    const unsigned blocks = static_cast<unsigned>((p.T + kRouteWarps - 1) / kRouteWarps);
    return host_launch(route_backward_kernel<L, NPL, FULL>, blocks, 32 * kRouteWarps, sizeof(float) * kRouteWarps * p.E, st, 0,
                       static_cast<const L *>(logits), static_cast<L *>(dlogits), p);
}

template <typename X, bool GATED>
gemm_status_t launch_quantize(const void *x, int8_t *q, const QuantParams &p, cudaStream_t st)
{
    const bool wide = aligned_to(x, 16) && aligned_to(q, 8) && p.ldx * static_cast<int64_t>(sizeof(X)) % 16 == 0 &&
                      p.ldq % 8 == 0 && p.K % 8 == 0;
    const int chunks = (p.K + 7) / 8;
    // Chunks a thread: small blocks, so that several share an SM and one's loads
    // overlap another's rounding. Blocks start at about one a nanosecond, so
    // many short rows share blocks, and rows of 257 .. 512 columns take a warp
    // each (16384 x 512: 17.1 us by a block a row, 9.4 by two warps a row, 8.2
    // by one); few rows spread out (128 x 301: 2.4 us by a warp, 1.9 by two).
    const bool many = p.M >= kQuantMany;
    const int ch = many && chunks > 32 && chunks <= 64 ? 2 : chunks <= 256 ? 1 : chunks <= 512 ? 2 : chunks <= 4 * kQuantMaxThreads ? 4 : 0;
    int threads = kQuantMaxThreads;
    if (ch > 0)
        threads = std::max(32, ((chunks + ch - 1) / ch + 31) / 32 * 32);
    const int rows = many ? std::max(1, kQuantShared / threads) : 1;
    const X *xp = static_cast<const X *>(x);
    const unsigned grid = static_cast<unsigned>((p.M + rows - 1) / rows);
#define G300_QUANT(W, C) return host_launch(quantize_kernel<X, GATED, W, C>, grid, dim3(threads, rows), 0, st, 0, xp, q, p)
#define G300_QUANT_CH(W)                                                                              \
    do {                                                                                              \
        if (ch == 1)                                                                                  \
            G300_QUANT(W, 1);                                                                         \
        else if (ch == 2)                                                                             \
            G300_QUANT(W, 2);                                                                         \
        else if (ch == 4)                                                                             \
            G300_QUANT(W, 4);                                                                         \
        else                                                                                          \
            G300_QUANT(W, 0);                                                                         \
    } while (0)
    if (wide)
        G300_QUANT_CH(true);
    else
        G300_QUANT_CH(false);
#undef G300_QUANT_CH
#undef G300_QUANT
}

}  // namespace

// ---------------------------------------------------------------- C ABI

extern "C" {

gemm_status_t gemm_route(int64_t T, int64_t E, const void *logits, gemm_out_t l_type, int64_t ldl, const float *bias,
                         int k, const gemm_route_t *route, float *weights, int32_t *ids, gemm_stream_t stream)
{
    gemm_route_t r;
    if (!valid_size(T) || !valid_type(l_type) || !route_rule(route, E, k, &r))
        return GEMM_ERR_INVALID_ARG;
    if (T == 0)
        return GEMM_OK;
    const int es = type_bytes(l_type);
    if (!logits || !weights || !ids || ldl < E || !valid_stride(ldl, es))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(logits, es) || !aligned_to(weights, 4) || !aligned_to(ids, 4) || !aligned_to(bias, 4))
        return GEMM_ERR_ALIGNMENT;
    RouteParams p = {};
    p.T = T;
    p.E = static_cast<int>(E);
    p.k = k;
    p.ldl = ldl;
    p.bias = bias;
    p.weights = weights;
    p.ids = ids;
    p.sigmoid = r.score == GEMM_ROUTE_SIGMOID;
    p.groups = r.groups;
    p.per = static_cast<int>(E) / r.groups;
    p.group_top = r.group_top;
    p.groups_kept = r.groups_kept;
    p.renorm = r.renormalize != 0;
    p.scale = r.scale;
    p.per_inv = p.per > 1 ? static_cast<unsigned int>(((uint64_t(1) << 32) + p.per - 1) / p.per) : 0u;
    for (p.group_lanes = 32; p.group_lanes * p.groups > 32;)
        p.group_lanes /= 2;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return with_type(l_type, [&](auto tag) {
        using L = decltype(tag);
        return E <= 32    ? launch_route<L, 1>(logits, p, st)
               : E <= 64  ? launch_route<L, 2>(logits, p, st)
               : E <= 128 ? launch_route<L, 4>(logits, p, st)
               : E <= 256 ? launch_route<L, 8>(logits, p, st)
               : E <= 512 ? launch_route<L, 16>(logits, p, st)
                          : launch_route<L, 32>(logits, p, st);
    });
}

gemm_status_t gemm_route_backward(int64_t T, int64_t E, const void *logits, gemm_out_t l_type, int64_t ldl, int k,
                                  const gemm_route_t *route, const int32_t *ids, const float *dweights, void *dlogits,
                                  int64_t lddl, gemm_stream_t stream)
{
    gemm_route_t r;
    if (!valid_size(T) || !valid_type(l_type) || !route_rule(route, E, k, &r))
        return GEMM_ERR_INVALID_ARG;
    if (T == 0)
        return GEMM_OK;
    const int es = type_bytes(l_type);
    if (!logits || !ids || !dweights || !dlogits || ldl < E || lddl < E || !valid_stride(ldl, es) ||
        !valid_stride(lddl, es))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(logits, es) || !aligned_to(dlogits, es) || !aligned_to(ids, 4) || !aligned_to(dweights, 4))
        return GEMM_ERR_ALIGNMENT;
    RouteGradParams p = {};
    p.T = T;
    p.E = static_cast<int>(E);
    p.k = k;
    p.ldl = ldl;
    p.lddl = lddl;
    p.ids = ids;
    p.dweights = dweights;
    p.sigmoid = r.score == GEMM_ROUTE_SIGMOID;
    p.renorm = r.renormalize != 0;
    p.scale = r.scale;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return with_type(l_type, [&](auto tag) {
        using L = decltype(tag);
        // the softmax over all experts, by the experts a lane holds; the others need none
        return p.sigmoid || p.renorm ? launch_route_backward<L, 1, false>(logits, dlogits, p, st)
               : E <= 64             ? launch_route_backward<L, 2, true>(logits, dlogits, p, st)
               : E <= 256            ? launch_route_backward<L, 8, true>(logits, dlogits, p, st)
               : E <= 512            ? launch_route_backward<L, 16, true>(logits, dlogits, p, st)
                                     : launch_route_backward<L, 32, true>(logits, dlogits, p, st);
    });
}

size_t gemm_route_plan_workspace_size(int64_t T, int64_t E, int k)
{
    if (T <= 0 || E < 1 || E > GEMM_ROUTE_MAX_EXPERTS || k < 1 || k > GEMM_ROUTE_MAX_K || T > kSizeLimit)
        return 0;
    const int blocks = plan_blocks(T * k);
    return blocks > 1 ? static_cast<size_t>(blocks) * static_cast<size_t>(E) * sizeof(int32_t) : 0;
}

gemm_status_t gemm_route_plan(int64_t T, int64_t E, int k, const int32_t *ids, int32_t *offsets, int32_t *slots,
                              int32_t *tokens, void *workspace, size_t workspace_bytes, gemm_stream_t stream)
{
    if (!valid_size(T) || E < 1 || E > GEMM_ROUTE_MAX_EXPERTS || k < 1 || k > GEMM_ROUTE_MAX_K || T * k > kSizeLimit)
        return GEMM_ERR_INVALID_ARG;
    if (!offsets || (T > 0 && (!ids || !slots || !tokens)))
        return GEMM_ERR_INVALID_ARG;
    const size_t need = gemm_route_plan_workspace_size(T, E, k);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(ids, 4) || !aligned_to(offsets, 4) || !aligned_to(slots, 4) || !aligned_to(tokens, 4) ||
        (need > 0 && !aligned_to(workspace, 4)))
        return GEMM_ERR_ALIGNMENT;
    const int64_t pairs = T * k;
    const int blocks = plan_blocks(pairs);
    const long long part = (pairs + blocks - 1) / blocks;
    const int warps = plan_warps(part, E);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int *counts = static_cast<int *>(workspace);
    if (blocks > 1) {
        const gemm_status_t c = host_launch(plan_count_kernel, static_cast<unsigned>(blocks), 32 * warps, E * sizeof(int), st, 0,
                                            ids, pairs, part, static_cast<int>(E), counts);
        if (c != GEMM_OK)
            return c;
    }
    // the scatter kernel starts while the counts are still being written, and
    // waits for them before it reads them
    return host_launch(plan_scatter_kernel, static_cast<unsigned>(blocks), 32 * warps,
                       static_cast<size_t>(warps + 2) * E * sizeof(int), st, 0, ids, pairs, part, static_cast<int>(E), k, counts,
                       offsets, slots, tokens);
}

gemm_status_t gemm_quantize_int8(int64_t M, int64_t K, const void *X, gemm_out_t x_type, int64_t x_rows, int64_t ldx,
                                 const int32_t *index, gemm_quant_t mode, int8_t *Q, int64_t ldq, float *scales,
                                 gemm_stream_t stream)
{
    if (!valid_size(M) || !valid_size(K) || !valid_size(x_rows) || !valid_type(x_type) ||
        (mode != GEMM_QUANT_PLAIN && mode != GEMM_QUANT_GATED))
        return GEMM_ERR_INVALID_ARG;
    if (M == 0)
        return GEMM_OK;
    const bool gated = mode == GEMM_QUANT_GATED;
    const int es = type_bytes(x_type);
    if (!scales || (!index && x_rows < M))
        return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (!Q || (x_rows > 0 && !X) || ldx < (gated ? 2 * K : K) || ldq < K || !valid_stride(ldx, es) ||
                  !valid_stride(ldq, 1)))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(X, es) || !aligned_to(index, 4) || !aligned_to(scales, 4))
        return GEMM_ERR_ALIGNMENT;
    if (!countable(K))
        return GEMM_ERR_UNSUPPORTED;
    QuantParams p = {};
    p.M = M;
    p.K = static_cast<int>(K);
    p.index = index;
    p.x_rows = x_rows;
    p.ldx = ldx;
    p.ldq = ldq;
    p.scales = scales;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return with_type(x_type, [&](auto tag) {
        using X_ = decltype(tag);
        return gated ? launch_quantize<X_, true>(X, Q, p, st) : launch_quantize<X_, false>(X, Q, p, st);
    });
}

gemm_status_t gemm_route_combine(int64_t T, int64_t N, int k, const void *Y, gemm_out_t y_type, int64_t y_rows,
                                 int64_t ldy, const int32_t *slots, const float *weights, void *D, gemm_out_t d_type,
                                 int64_t ldd, gemm_stream_t stream)
{
    if (!valid_size(T) || !valid_size(N) || !valid_size(y_rows) || k < 1 || k > GEMM_ROUTE_MAX_K ||
        !valid_type(y_type) || !valid_type(d_type))
        return GEMM_ERR_INVALID_ARG;
    if (T == 0 || N == 0)
        return GEMM_OK;
    const int ey = type_bytes(y_type), ed = type_bytes(d_type);
    if ((y_rows > 0 && !Y) || !slots || !weights || !D || ldy < N || ldd < N || !valid_stride(ldy, ey) ||
        !valid_stride(ldd, ed))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(Y, ey) || !aligned_to(D, ed) || !aligned_to(slots, 4) || !aligned_to(weights, 4))
        return GEMM_ERR_ALIGNMENT;
    const int64_t col_blocks = (N + 8 * kCombineThreads - 1) / (8 * kCombineThreads);
    if (!countable(N) || col_blocks * T > kSizeLimit)
        return GEMM_ERR_UNSUPPORTED;
    CombineParams p = {};
    p.T = T;
    p.N = static_cast<int>(N);
    p.k = k;
    p.y_rows = y_rows;
    p.ldy = ldy;
    p.ldd = ldd;
    p.slots = slots;
    p.weights = weights;
    const bool wide = N % 8 == 0 && aligned_to(Y, 16) && aligned_to(D, 16) && ldy * ey % 16 == 0 && ldd * ed % 16 == 0;
    const unsigned grid = static_cast<unsigned>(col_blocks * T);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return with_type(y_type, [&](auto ytag) {
        using Y_ = decltype(ytag);
        return with_type(d_type, [&](auto dtag) {
            using D_ = decltype(dtag);
            const Y_ *yp = static_cast<const Y_ *>(Y);
            D_ *dp = static_cast<D_ *>(D);
            return host_launch(wide ? combine_kernel<Y_, D_, true> : combine_kernel<Y_, D_, false>, grid, kCombineThreads, 0, st, 0,
                               yp, dp, p, static_cast<int>(col_blocks));
        });
    });
}

gemm_status_t gemm_route_combine_backward(int64_t T, int64_t N, int k, const void *dD, gemm_out_t d_type, int64_t lddd,
                                          const void *Y, gemm_out_t y_type, int64_t y_rows, int64_t ldy,
                                          const int32_t *slots, const float *weights, void *dY, int64_t lddy,
                                          float *dweights, gemm_stream_t stream)
{
    if (!valid_size(T) || !valid_size(N) || !valid_size(y_rows) || k < 1 || k > GEMM_ROUTE_MAX_K ||
        !valid_type(y_type) || !valid_type(d_type) || T * k > kSizeLimit)
        return GEMM_ERR_INVALID_ARG;
    if (T == 0)
        return GEMM_OK;
    const int ey = type_bytes(y_type), ed = type_bytes(d_type);
    if (!slots || !weights || !dweights || (N > 0 && !dD) || (N > 0 && y_rows > 0 && (!Y || !dY)) || lddd < N ||
        ldy < N || lddy < N || !valid_stride(lddd, ed) || !valid_stride(ldy, ey) || !valid_stride(lddy, ey))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(dD, ed) || !aligned_to(Y, ey) || !aligned_to(dY, ey) || !aligned_to(slots, 4) ||
        !aligned_to(weights, 4) || !aligned_to(dweights, 4))
        return GEMM_ERR_ALIGNMENT;
    if (!countable(N))
        return GEMM_ERR_UNSUPPORTED;
    CombineGradParams p = {};
    p.T = T;
    p.N = static_cast<int>(N);
    p.k = k;
    p.y_rows = y_rows;
    p.ldy = ldy;
    p.lddy = lddy;
    p.lddd = lddd;
    p.slots = slots;
    p.weights = weights;
    p.dweights = dweights;
    const bool wide = N % 8 == 0 && aligned_to(dD, 16) && aligned_to(Y, 16) && aligned_to(dY, 16) &&
                      lddd * ed % 16 == 0 && ldy * ey % 16 == 0 && lddy * ey % 16 == 0;
    const bool shared = combine_grad_shared(T * k, N);
    const unsigned grid = static_cast<unsigned>(shared ? T * k : (T * k + kCombineGradWarps - 1) / kCombineGradWarps);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return with_type(y_type, [&](auto ytag) {
        using Y_ = decltype(ytag);
        return with_type(d_type, [&](auto dtag) {
            using D_ = decltype(dtag);
            const D_ *gp = static_cast<const D_ *>(dD);
            const Y_ *yp = static_cast<const Y_ *>(Y);
            Y_ *op = static_cast<Y_ *>(dY);
            return host_launch(shared ? wide ? combine_backward_kernel<Y_, D_, true, true> : combine_backward_kernel<Y_, D_, false, true>
                               : wide ? combine_backward_kernel<Y_, D_, true, false>
                                      : combine_backward_kernel<Y_, D_, false, false>,
                               grid, 32 * kCombineGradWarps, 0, st, 0, gp, yp, op, p);
        });
    });
}

}  // extern "C"
