// The balance loss of a router and its counts per expert, with the gradient of
// its logits. Contracts are in include/gemm_gb300.h.
//
//   n_e = choices of e among the n live tokens of a sequence, P_e = mean of p_te
//   loss = E sum_e n_e / (k n) P_e
//   c_e = dloss E n_e / (k n^2);  softmax: dl = p (c - sum p c),
//   sigmoid scores over their sum, p = s / Z: dl = s (1 - s) / Z (c - sum p c)
//
// The tokens are cut into equal parts, one for each block, whatever the
// sequences' lengths. A part and a sequence that meet have a slot of the
// workspace, part + sequence (one of the two grows from each meeting to the
// next), where the block leaves its counts and sums; a sequence's slots are
// added in their order, by a second launch.
//
// Measured as a call: forward of 16384 tokens, 256 experts, k 8, sigmoid scores,
// fp32 logits 10.3 us (2.6 by its bytes; two launches that wait for one another,
// each a chain of loads and sums), backward of 16384 tokens, 64 experts, k 6 in
// 7 sequences 6.3 us (0.7), near what a call takes on the host.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gemm_gb300.h"
#include "elements.cuh"
#include "host.h"
#include "ptx.cuh"

using namespace g300;

namespace {

struct BalanceParams {
    long long T, S;
    int E, k, sigmoid;
    long long ldl, lddl;
    const int *ids, *offsets;
    int *counts, *tokens;
    float *means, *losses;
    long long part;  // tokens of a block
    int blocks;
    int alone;       // the only block finishes the sequences itself
    int *slot_counts, *slot_tokens;
    float *slot_sums;
    long long ld_slot;
    int join_ctas;
    const float *dlosses;
    int accumulate;
};

// The tokens of sequence s, inside 0..T.
struct Sequence {
    long long lo, hi;
};

__device__ __forceinline__ Sequence sequence(const BalanceParams &p, long long s)
{
    if (!p.offsets)
        return {0, p.T};
    Sequence q;
    q.lo = min(max(static_cast<long long>(__ldcg(p.offsets + s)), 0ll), p.T);
    q.hi = min(max(static_cast<long long>(__ldcg(p.offsets + s + 1)), q.lo), p.T);
    return q;
}

// The last sequence that begins at token t or before it (0 if none does).
__device__ __forceinline__ long long sequence_of(const BalanceParams &p, long long t)
{
    if (!p.offsets)
        return 0;
    long long lo = 0, hi = p.S - 1;
    while (lo < hi) {
        const long long mid = (lo + hi + 1) / 2;
        if (__ldcg(p.offsets + mid) <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// The logits of a token, expert lane + 32 i in x[i].
template <typename L, int NPL>
__device__ __forceinline__ void load_logits(const L *row, int E, int lane, float (&x)[NPL])
{
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        x[i] = e < E ? to_float(row[e]) : -INFINITY;
    }
}

// e^x and 1 / x by the special-function unit, to within 2^-21 for the logits that
// a router has (|x| < 10; 2^-22 and |x| 2^-24 of the product with log2 e): sums
// over tokens are what they are for. By expf and correctly rounded reciprocals
// 16384 x 256 took 13.8 us instead of 11.3.
__device__ __forceinline__ float fast_exp(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

__device__ __forceinline__ float fast_inverse(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Scores of a token: p unnormalised, and the factor that normalises it.
template <int NPL>
__device__ __forceinline__ float scores(bool sigmoid, const float (&x)[NPL], float (&v)[NPL])
{
    float total = 0.0f;
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            v[i] = fast_inverse(1.0f + fast_exp(-x[i]));  // -inf: 1 / inf
    } else {
        float top = x[0];
#pragma unroll
        for (int i = 1; i < NPL; ++i)
            top = fmaxf(top, x[i]);
        top = warp_max(top);
        if (top == -INFINITY)
            top = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            v[i] = fast_exp(x[i] - top);
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        total += v[i];
    total = warp_sum(total);
    return fast_inverse(total == 0.0f ? 1.0f : total);
}

// Warps of a block: their sums of all experts take 32 KB of shared memory.
template <int NPL>
constexpr int kBalanceWarps = NPL <= 8 ? 32 : NPL == 16 ? 16 : 8;

// Counts, means and loss of one sequence from sums and counts in shared memory.
__device__ void balance_finish(const BalanceParams &p, long long s, const float *sums, const int *counts, int n)
{
    __shared__ float warp_part[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = static_cast<int>(blockDim.x >> 5);
    const float live = static_cast<float>(max(n, 1));
    float loss = 0.0f;
    for (int e = tid; e < p.E; e += blockDim.x) {
        const float mean = __fdiv_rn(sums[e], live);
        const int c = counts[e];
        p.counts[s * p.E + e] = c;
        p.means[s * p.E + e] = mean;
        loss = fmaf(__fdiv_rn(static_cast<float>(c), static_cast<float>(p.k) * live), mean, loss);
    }
    loss = warp_sum(loss);
    if (lane == 0)
        warp_part[warp] = loss;
    __syncthreads();
    if (tid == 0) {
        loss = 0.0f;
        for (int w = 0; w < warps; ++w)
            loss += warp_part[w];
        p.losses[s] = static_cast<float>(p.E) * loss;
        p.tokens[s] = n;
    }
    __syncthreads();
}

// One block's part of the tokens, one warp a token.
template <typename L, int NPL>
__global__ void __launch_bounds__(32 * kBalanceWarps<NPL>) balance_kernel(const L *logits, const BalanceParams p)
{
    constexpr int WARPS = kBalanceWarps<NPL>;
    __shared__ float sums[WARPS][32 * NPL];
    __shared__ int counts[32 * NPL], tokens;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_start();
    const long long lo = blockIdx.x * p.part, hi = min(lo + p.part, p.T);
    // up to 31 sequences: each lane has the end of one
    const bool few = p.offsets && p.S < 32;
    const long long mine_end = few && lane <= p.S ? min(max(static_cast<long long>(__ldcg(p.offsets + lane)), 0ll), p.T) : p.T;
    long long s = 0;
    if (!p.alone)
        s = few ? max(0, __popc(__ballot_sync(0xffffffffu, lane < p.S && mine_end <= lo)) - 1) : sequence_of(p, lo);
    for (; s < p.S; ++s) {
        Sequence q;
        if (few) {
            q.lo = __shfl_sync(0xffffffffu, mine_end, static_cast<int>(s));
            q.hi = max(q.lo, __shfl_sync(0xffffffffu, mine_end, static_cast<int>(s) + 1));
        } else {
            q = sequence(p, s);
        }
        if (q.lo >= hi && !p.alone)
            return;
        const long long a = max(lo, q.lo), b = min(hi, q.hi);
        if (a >= b && !p.alone) {
            if (!few)  // past the empty ones that begin there too, however many
                s = max(s, sequence_of(p, max(lo, q.hi)) - 1);
            continue;
        }
        for (int e = tid; e < 32 * NPL; e += 32 * WARPS)
            counts[e] = 0;
        if (tid == 0)
            tokens = 0;
        __syncthreads();
        float sum[NPL] = {};
        int mine = 0;
        // a token's logits and ids are asked for before the one before it is worked on
        auto id_of = [&](long long t) { return lane < p.k && t < b ? p.ids[t * p.k + lane] : -1; };
        float x[NPL];
        int id = id_of(a + warp);
        if (a + warp < b)
            load_logits<L, NPL>(logits + (a + warp) * p.ldl, p.E, lane, x);
        for (long long t = a + warp; t < b; t += WARPS) {
            float x_next[NPL];
            const int id_next = id_of(t + WARPS);
            if (t + WARPS < b)
                load_logits<L, NPL>(logits + (t + WARPS) * p.ldl, p.E, lane, x_next);
            float v[NPL];
            const float inv = scores<NPL>(p.sigmoid != 0, x, v);
            const bool chosen = id >= 0 && id < p.E;
            if (__any_sync(0xffffffffu, chosen)) {
                ++mine;
                if (chosen)
                    atomicAdd(&counts[id], 1);  // a count: the order of the additions does not show
#pragma unroll
                for (int i = 0; i < NPL; ++i)
                    sum[i] = fmaf(v[i], inv, sum[i]);
            }
            id = id_next;
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                x[i] = x_next[i];
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            sums[warp][lane + 32 * i] = sum[i];
        if (lane == 0)
            atomicAdd(&tokens, mine);
        __syncthreads();
        for (int e = tid; e < p.E; e += 32 * WARPS) {
            float total = sums[0][e];
#pragma unroll
            for (int w = 1; w < WARPS; ++w)
                total += sums[w][e];
            sums[0][e] = total;
        }
        __syncthreads();
        if (p.alone) {
            balance_finish(p, s, sums[0], counts, tokens);
        } else {
            const long long slot = blockIdx.x + s;
            for (int e = tid; e < p.E; e += 32 * WARPS) {
                p.slot_sums[slot * p.ld_slot + e] = sums[0][e];
                p.slot_counts[slot * p.ld_slot + e] = counts[e];
            }
            if (tid == 0)
                p.slot_tokens[slot] = tokens;
            __syncthreads();
        }
    }
}

// Parts of the tokens: one for each SM of the GPU this is built for (16384 tokens
// in 500 sequences 28 us; in a part for each sequence 50). A block takes the
// sequences that it meets one after another, in 1 to 2 us each, so that few tokens
// are cut into parts as long as a sequence (51 tokens in 16 sequences took 20.8 us
// by parts of 32, 7.8 by 4; 2048 in 64 took 12.2 by 32 and 19.9 by 14).
constexpr int kBalanceBlocks = 152;

constexpr int kJoinThreads = 512;
constexpr int kJoinGroups = 64;      // at most
constexpr int kJoinMaxCtas = 8;      // of a cluster, which has a sequence: each has a share of the experts

// CTAs that share a sequence's experts: fewer where there are many sequences (2048
// tokens of 256 experts in 200 sequences 32 us by 8 CTAs each, 19.6 by one; 16384
// of 64 experts in 500 28 by 2, 23.9 by one), but a thread for each expert.
inline int join_ctas(int64_t E, int64_t S)
{
    int n = E <= 32 ? 1 : E <= 64 ? 2 : E <= 128 ? 4 : kJoinMaxCtas;
    while (n > 1 && S * n > 2 * kBalanceBlocks && (E + 3) / 4 * 4 <= kJoinThreads * (n / 2))
        n /= 2;
    return n;
}

// A sequence's slots, added by groups of threads that take every so-manieth
// one; then the groups in their order; then the loss over the cluster's CTAs.
__global__ void __launch_bounds__(kJoinThreads) balance_join_kernel(const BalanceParams p)
{
    __shared__ float4 sums[kJoinThreads];
    __shared__ int4 counts[kJoinThreads];
    __shared__ float warp_loss[kJoinThreads / 32], cta_loss[kJoinMaxCtas];
    __shared__ int tokens;
    const int tid = threadIdx.x, ctas = p.join_ctas, cta = static_cast<int>(blockIdx.x) % ctas;
    const long long s = blockIdx.x / ctas;
    // this CTA's experts: whole words of four
    const int per = (static_cast<int>(p.ld_slot) / 4 + ctas - 1) / ctas, w0 = cta * per;
    const int words = max(0, min(per, static_cast<int>(p.ld_slot) / 4 - w0));
    const int groups = words ? min(kJoinThreads / words, kJoinGroups) : 0;
    const int group = words ? tid / words : 0, word = words ? tid - group * words : 0;
    if (tid == 0)
        tokens = 0;
    if (ctas > 1)
        cluster_arrive();  // this CTA has started: the others may write its shared memory
    grid_start();
    __syncthreads();
    const Sequence q = sequence(p, s);
    long long first = 0, end = 0;
    if (q.lo < q.hi) {
        first = q.lo / p.part + s;
        end = (q.hi - 1) / p.part + s + 1;
    }
    int n = 0;
    for (long long i = first + tid; i < end; i += kJoinThreads)
        n += __ldcg(p.slot_tokens + i);
    if (group < groups) {
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        int4 c = make_int4(0, 0, 0, 0);
#pragma unroll 4
        for (long long i = first + group; i < end; i += groups) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.slot_sums + i * p.ld_slot) + w0 + word);
            const int4 k = __ldcg(reinterpret_cast<const int4 *>(p.slot_counts + i * p.ld_slot) + w0 + word);
            f.x += v.x;
            f.y += v.y;
            f.z += v.z;
            f.w += v.w;
            c.x += k.x;
            c.y += k.y;
            c.z += k.z;
            c.w += k.w;
        }
        sums[tid] = f;
        counts[tid] = c;
    }
    if (n)
        atomicAdd(&tokens, n);
    __syncthreads();
    const float live = static_cast<float>(max(tokens, 1));
    float loss = 0.0f;
    const int e = 4 * w0 + tid;
    if (tid < 4 * words && e < p.E) {
        float f = 0.0f;
        int c = 0;
#pragma unroll 8
        for (int g = 0; g < groups; ++g) {
            f += reinterpret_cast<const float *>(sums)[4 * words * g + tid];
            c += reinterpret_cast<const int *>(counts)[4 * words * g + tid];
        }
        const float mean = __fdiv_rn(f, live);
        p.counts[s * p.E + e] = c;
        p.means[s * p.E + e] = mean;
        loss = __fdiv_rn(static_cast<float>(c), static_cast<float>(p.k) * live) * mean;
    }
    loss = warp_sum(loss);
    if ((tid & 31) == 0)
        warp_loss[tid >> 5] = loss;
    __syncthreads();
    if (ctas > 1)
        cluster_wait();  // the first CTA has started
    if (tid == 0) {
        loss = 0.0f;
        for (int w = 0; w < kJoinThreads / 32; ++w)
            loss += warp_loss[w];
        if (ctas == 1)
            cta_loss[0] = loss;
        else  // to the first CTA of the cluster
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&cta_loss[cta]), 0)), "f"(loss) : "memory");
    }
    if (ctas > 1) {
        __syncwarp();
        cluster_sync_all();
    }
    if (cta == 0 && tid == 0) {
        loss = 0.0f;
        for (int i = 0; i < ctas; ++i)
            loss += cta_loss[i];
        p.losses[s] = static_cast<float>(p.E) * loss;
        p.tokens[s] = tokens;
    }
}

constexpr int kBalanceGradWarps = 8;

// Tokens of a warp: neighbours, which mostly share a sequence, and whose logits
// are all asked for at the start.
template <int NPL>
constexpr int kBalanceGradRun = NPL <= 2 ? 4 : NPL <= 8 ? 2 : 1;

// One warp a token: its scores, their mean gradient, and the logits' gradients.
template <typename L, int NPL>
__global__ void __launch_bounds__(32 * kBalanceGradWarps) balance_backward_kernel(const L *logits, L *dlogits, const BalanceParams p)
{
    constexpr int RUN = kBalanceGradRun<NPL>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t0 = (static_cast<long long>(blockIdx.x) * kBalanceGradWarps + warp) * RUN;
    grid_start();
    if (t0 >= p.T)
        return;
    float x[RUN][NPL];
    int id[RUN];
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
        const bool have = t0 + r < p.T;
        id[r] = lane < p.k && have ? p.ids[(t0 + r) * p.k + lane] : -1;
        load_logits<L, NPL>(logits + (have ? t0 + r : t0) * p.ldl, p.E, lane, x[r]);
    }
    // up to 31 sequences: each lane has the end of one
    const bool few = p.offsets && p.S < 32;
    long long mine = 0;
    if (few)
        mine = lane <= p.S ? min(max(static_cast<long long>(__ldcg(p.offsets + lane)), 0ll), p.T) : p.T;
    long long s = -1;
    Sequence q = {0, 0};
    float c[NPL];
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
        const long long t = t0 + r;
        if (t >= p.T)
            return;
        if (s < 0 || t >= q.hi) {
            if (few) {
                s = max(0, __popc(__ballot_sync(0xffffffffu, lane < p.S && mine <= t)) - 1);
                q.lo = __shfl_sync(0xffffffffu, mine, static_cast<int>(s));
                q.hi = max(q.lo, __shfl_sync(0xffffffffu, mine, static_cast<int>(s) + 1));
            } else {
                s = sequence_of(p, t);
                q = sequence(p, s);
            }
            const float n = static_cast<float>(max(__ldcg(p.tokens + s), 1));
            const float by = __fdiv_rn(__fdiv_rn(__ldcg(p.dlosses + s) * static_cast<float>(p.E), static_cast<float>(p.k) * n), n);
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const int e = lane + 32 * i;
                c[i] = e < p.E ? by * static_cast<float>(__ldcg(p.counts + s * p.E + e)) : 0.0f;
            }
        }
        if (t < q.lo || t >= q.hi)
            continue;  // a token of no sequence
        const bool live = __any_sync(0xffffffffu, id[r] >= 0 && id[r] < p.E);
        if (!live && p.accumulate)
            continue;
        L *out = dlogits + t * p.lddl;
        float d[NPL] = {};
        if (live) {
            const float inv = scores<NPL>(p.sigmoid != 0, x[r], d);
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                dot = fmaf(d[i] * inv, c[i], dot);
            dot = warp_sum(dot);
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                d[i] = d[i] * inv * (c[i] - dot);
                if (p.sigmoid)
                    d[i] *= fast_inverse(1.0f + fast_exp(x[r][i]));  // 1 - s without its cancellation
            }
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 32 * i;
            if (e < p.E)
                out[e] = from_float<L>(p.accumulate ? to_float(out[e]) + d[i] : d[i]);
        }
    }
}

// ---------------------------------------------------------------- host

constexpr int kBalanceLeastPart = 4, kBalancePart = 32;
// Sequences that one block takes alone, in one launch: 32 tokens and 64 experts
// in two sequences 4.9 us (5.9 by two launches), in three 6.9 (5.9 to 7.4).
constexpr int kBalanceAlone = 2;

struct BalancePlan {
    int blocks;
    bool alone;
    int64_t part, ld;
    size_t counts, tokens, bytes;  // offsets; the sums come first
};

BalancePlan balance_plan(int64_t T, int64_t E, int64_t S)
{
    BalancePlan b = {};
    b.part = S <= kBalanceAlone && T <= kBalancePart ? T : std::clamp<int64_t>(T / std::max<int64_t>(S, 1), kBalanceLeastPart, kBalancePart);
    b.part = std::max(b.part, (T + kBalanceBlocks - 1) / kBalanceBlocks);
    b.blocks = static_cast<int>((T + b.part - 1) / b.part);
    b.ld = (E + 3) / 4 * 4;
    b.alone = b.blocks <= 1 && S <= kBalanceAlone;
    if (b.alone)
        return b;
    const int64_t slots = b.blocks + S - 1;
    const size_t one = static_cast<size_t>((slots * b.ld * 4 + 255) / 256 * 256);
    b.counts = one;
    b.tokens = 2 * one;
    b.bytes = 2 * one + static_cast<size_t>((slots * 4 + 255) / 256 * 256);
    return b;
}

// Room for T tokens and for fewer. Parts of one length are more for more tokens;
// they get longer by one where the tokens reach another multiple of the sequences
// or of the blocks. (Fewer sequences never have shorter parts.)
size_t balance_bytes(int64_t T, int64_t E, int64_t S)
{
    size_t most = balance_plan(T, E, S).bytes;
    for (int64_t part = kBalanceLeastPart; part <= kBalancePart; ++part)
        for (const int64_t last : {(part + 1) * S - 1, part * kBalanceBlocks})
            if (last < T)
                most = std::max(most, balance_plan(last, E, S).bytes);
    return most;
}

// What both calls check, and the parameters that they share.
gemm_status_t check_balance(int64_t T, int64_t E, const void *logits, int l_type, int64_t ldl, int k, const gemm_route_t *route,
                            const int32_t *ids, int64_t S, const int32_t *offsets, BalanceParams *p)
{
    const int score = route ? route->score : GEMM_ROUTE_SOFTMAX;
    if (!valid_size(T) || !valid_type(l_type) || E < 1 || E > GEMM_ROUTE_MAX_EXPERTS || k < 1 || k > GEMM_ROUTE_MAX_K || k > E ||
        (score != GEMM_ROUTE_SOFTMAX && score != GEMM_ROUTE_SIGMOID) || S < 0 || S > kSizeLimit / std::max<int64_t>(E, 8) || (!offsets && S != 1))
        return GEMM_ERR_INVALID_ARG;
    const int es = type_bytes(l_type);
    if (T > 0 && (!logits || !ids || ldl < E || !valid_stride(ldl, es)))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(logits, es) || !aligned_to(ids, 4) || !aligned_to(offsets, 4))
        return GEMM_ERR_ALIGNMENT;
    *p = BalanceParams{};
    p->T = T;
    p->S = S;
    p->E = static_cast<int>(E);
    p->k = k;
    p->sigmoid = score == GEMM_ROUTE_SIGMOID;
    p->ldl = ldl;
    p->ids = ids;
    p->offsets = offsets;
    return GEMM_OK;
}

template <typename L, int NPL>
gemm_status_t launch_balance(const void *logits, const BalanceParams &p, cudaStream_t st)
{
    return host_launch(balance_kernel<L, NPL>, static_cast<unsigned>(p.blocks), 32 * kBalanceWarps<NPL>, 0, st, 0,
                       static_cast<const L *>(logits), p);
}

template <typename L, int NPL>
gemm_status_t launch_balance_backward(const void *logits, void *dlogits, const BalanceParams &p, cudaStream_t st)
{
    const int64_t tokens = kBalanceGradWarps * kBalanceGradRun<NPL>;
    return host_launch(balance_backward_kernel<L, NPL>, static_cast<unsigned>((p.T + tokens - 1) / tokens), 32 * kBalanceGradWarps, 0, st, 0,
                       static_cast<const L *>(logits), static_cast<L *>(dlogits), p);
}

}  // namespace

// ---------------------------------------------------------------- C ABI

extern "C" {

size_t gemm_route_balance_workspace_size(int64_t T, int64_t E, int64_t S)
{
    if (T < 1 || T > kSizeLimit || E < 1 || E > GEMM_ROUTE_MAX_EXPERTS || S < 1 || S > kSizeLimit / std::max<int64_t>(E, 8))
        return 0;
    return balance_bytes(T, E, S);
}

gemm_status_t gemm_route_balance(int64_t T, int64_t E, const void *logits, gemm_out_t l_type, int64_t ldl, int k, const gemm_route_t *route,
                                 const int32_t *ids, int64_t S, const int32_t *offsets, int32_t *counts, int32_t *tokens, float *means,
                                 float *losses, void *workspace, size_t workspace_bytes, gemm_stream_t stream)
{
    BalanceParams p;
    gemm_status_t s = check_balance(T, E, logits, l_type, ldl, k, route, ids, S, offsets, &p);
    if (s != GEMM_OK || S == 0)
        return s;
    if (!counts || !tokens || !means || !losses)
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(counts, 4) || !aligned_to(tokens, 4) || !aligned_to(means, 4) || !aligned_to(losses, 4))
        return GEMM_ERR_ALIGNMENT;
    BalancePlan b = balance_plan(std::max<int64_t>(T, 1), E, S);
    if (T == 0) {  // the second launch alone writes the zeros, from no slots
        b.bytes = 0;
        b.alone = false;
        b.ld = (E + 3) / 4 * 4;
    }
    if (b.bytes > 0 && (!workspace || workspace_bytes < b.bytes))
        return GEMM_ERR_INVALID_ARG;
    if (b.bytes > 0 && !aligned_to(workspace, 16))
        return GEMM_ERR_ALIGNMENT;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.counts = counts;
    p.tokens = tokens;
    p.means = means;
    p.losses = losses;
    p.part = b.part;
    p.blocks = b.blocks;
    p.alone = b.alone;
    p.slot_sums = reinterpret_cast<float *>(ws);
    p.slot_counts = reinterpret_cast<int *>(ws + b.counts);
    p.slot_tokens = reinterpret_cast<int *>(ws + b.tokens);
    p.ld_slot = b.ld;
    p.join_ctas = join_ctas(E, S);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    s = T == 0 ? GEMM_OK : with_type(l_type, [&](auto tag) {
        using L = decltype(tag);
        return E <= 64    ? launch_balance<L, 2>(logits, p, st)
               : E <= 128 ? launch_balance<L, 4>(logits, p, st)
               : E <= 256 ? launch_balance<L, 8>(logits, p, st)
               : E <= 512 ? launch_balance<L, 16>(logits, p, st)
                          : launch_balance<L, 32>(logits, p, st);
    });
    if (s != GEMM_OK || b.alone)
        return s;
    return host_launch(balance_join_kernel, static_cast<unsigned>(S * p.join_ctas), kJoinThreads, 0, st,
                       p.join_ctas > 1 ? static_cast<unsigned>(p.join_ctas) : 0u, p);
}

gemm_status_t gemm_route_balance_backward(int64_t T, int64_t E, const void *logits, gemm_out_t l_type, int64_t ldl, int k,
                                          const gemm_route_t *route, const int32_t *ids, int64_t S, const int32_t *offsets,
                                          const int32_t *counts, const int32_t *tokens, const float *dlosses, void *dlogits, int64_t lddl,
                                          int accumulate, gemm_stream_t stream)
{
    BalanceParams p;
    const gemm_status_t s = check_balance(T, E, logits, l_type, ldl, k, route, ids, S, offsets, &p);
    if (s != GEMM_OK || S == 0 || T == 0)
        return s;
    const int es = type_bytes(l_type);
    if (!counts || !tokens || !dlosses || !dlogits || lddl < E || !valid_stride(lddl, es))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(counts, 4) || !aligned_to(tokens, 4) || !aligned_to(dlosses, 4) || !aligned_to(dlogits, es))
        return GEMM_ERR_ALIGNMENT;
    p.counts = const_cast<int *>(counts);
    p.tokens = const_cast<int *>(tokens);
    p.dlosses = dlosses;
    p.lddl = lddl;
    p.accumulate = accumulate != 0;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return with_type(l_type, [&](auto tag) {
        using L = decltype(tag);
        return E <= 64    ? launch_balance_backward<L, 2>(logits, dlogits, p, st)
               : E <= 128 ? launch_balance_backward<L, 4>(logits, dlogits, p, st)
               : E <= 256 ? launch_balance_backward<L, 8>(logits, dlogits, p, st)
               : E <= 512 ? launch_balance_backward<L, 16>(logits, dlogits, p, st)
                          : launch_balance_backward<L, 32>(logits, dlogits, p, st);
    });
}

}  // extern "C"
