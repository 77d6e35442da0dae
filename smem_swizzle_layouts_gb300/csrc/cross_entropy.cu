// Softmax cross entropy of a linear head, in pieces of the vocabulary and
// without keeping the logits, with its gradients. Contracts are in
// include/gemm_gb300.h.
//
//   l = X W^T            T tokens, V words, K features; fp32 in TMEM only
//   lse_t = log sum_v exp(l_tv),   loss_t = lse_t - l_{t, y_t}
//   dl_tv = exp(l_tv - lse_t) (dloss_t + dlse_t) - [v = y_t] dloss_t
//   dX = dl W,   dW = dl^T X
//
// One kernel template does the four products, by what its epilogue does with a
// tile of the accumulator: the running maximum and sum of a softmax (forward),
// dl rounded to the inputs' type (backward, a piece of the vocabulary at a
// time into the workspace: the logits are computed a second time, 2 T V K of
// the 6 T V K operations of the backward pass), or the gradients themselves.
// Backward, one launch has up to three products: a piece's dX and dW, and the
// next piece's dl, whose units fill what the others' rounds leave of the grid
// (4096 x 32768 x 4096: 1958 us instead of 2234 by a launch for each, before
// the logits were summed in parts of K). One or two tokens have a kernel of
// their own below.
//
// Many tokens are bound by the tensor cores, whose rate the power limit holds:
// 8192 x 65536 x 4096 forward took 2409 to 2551 us (1.8 PFLOP/s; at the measured
// peaks 2280 in a burst, 2500 sustained), 4096 x 32768 x 4096 backward
// 1916 to 2003 (1710, 1875). Few are bound by the weights' bytes: 1 x 131072 x
// 4096 in 159 to 163 us, at the rate of a copy. Small K is bound by the epilogue, an exponential and some
// additions for each logit against K products, and backward by dl's bytes: 8192 x
// 32768 x 256 forward 112 to 118 us of 71, backward 352 to 365 of 214.
//
// Roles, barriers and waits are those of gemm_kernel.cuh (whose operand
// geometry, descriptors and bounded waits are used here); the tiles' widths,
// stage depths and splits of K are arguments, so that each product has the
// tiles that fill the SMs best.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/gemm_gb300.h"
#include "elements.cuh"
#include "gemm_kernel.cuh"
#include "host.h"
#include "launch.cuh"

using namespace g300;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What a launch of the kernel does: the forward product; gradients; gradients
// with dl whose sums over K are taken in parts.
enum : int { kForward = 0, kBackward = 1, kBackwardParts = 2 };

// Epilogue warps: a lane quarter each, and a half or (a pair's softmax) a quarter
// of the columns. The softmax has no staging buffers, and while some of its 16
// warps wait for TMEM others have work: 7252 x 118755 x 128 forward 346 us (384
// by 8), 8192 x 32768 x 256 112 (123); 2048 x 32768 x 1024 78.7 (77.3). A single
// CTA's few rows leave most warps without any: 1 x 131072 x 4096 167 (157). (By 16
// a thread has 96 registers, and 32 bytes of it lie in memory.)
template <int CG, int MODE>
constexpr int kHeadWarps = CG == 2 && MODE == kForward ? 16 : 8;
// Before them the producer and the issuer. Where dl is made of parts, a thread
// holds 128 sums beside what it packs: two idle warps make the first four a
// warpgroup that leaves registers to the epilogue's (without that the sums went
// through memory: 4096 x 32768 x 4096 2070 to 2370 us, now 1918). Such launches
// have a kernel of their own, as that code in one with the others slowed them down
// (8192 x 32768 x 256 backward 388 us instead of 365).
template <int MODE>
constexpr int kHeadFirstWarp = MODE == kBackwardParts ? 4 : 2;
template <int CG, int MODE>
constexpr int kHeadThreads = 32 * (kHeadFirstWarp<MODE> + kHeadWarps<CG, MODE>);
constexpr int kBackLaunchRegs = 168, kBackIssueRegs = 56, kBackEpiRegs = 224;
static_assert(128 * kBackIssueRegs + 32 * kHeadWarps<2, kBackwardParts> * kBackEpiRegs <= kHeadThreads<2, kBackwardParts> * kBackLaunchRegs &&
                  kHeadThreads<2, kBackwardParts> * kBackLaunchRegs <= 65536,
              "the shares add up to no more than the block is launched with");
constexpr int kHeadMaxStages = 12;
constexpr int kAccStride = 256;                    // TMEM columns from one accumulator to the next
constexpr int kHeadSmem = 232448 - 1024;           // less the slack that rounds the base up to 1024 bytes

// Elements of K that the tensor cores sum for a logit before the sum is added to
// the others in registers. Their additions truncate (every 16 elements, to the
// accumulator's 24 bits), which moves a logit towards 0 by up to half a part in
// 2^24 for each. Relative error of the losses, and time, of 8192 tokens, 65536
// words and K = 4096 by parts of 256, 512, 1024 and all of K: 0.9e-7 (2516 us),
// 1.7e-7 (2409), 3.3e-7 (2370), 1.4e-6 (2387). A single CTA's tiles wait for the
// weights: their parts of 256 take as long (77 x 50001 x 2001: 45.1 us by 512,
// 45.6 by 256, 46.3 by 128). Backward the logits are summed in the same parts, so
// that exp(l - lse) is 1 where it should be: with all of K in one part a target's
// dl of 3e-10 came out as 4e-4 (K = 4096, a logit of 30) and 2e-3 (16384); with
// these parts it is 1e-6, for 2 to 4 % of the time (4096 x 32768 x 4096 1918
// us instead of 1876, 777 x 50001 x 1001 238 instead of 230, 128 x 131072 x 2048
// 330 both ways). The gradients of one or two tokens may be without tiles, by
// sums that round, where the forward pass's error does not cancel: theirs
// are the smallest parts (1 x 131072 x 4096: 158.1 us by 512, 159.5 by 128; dl 3e-5
// and 4e-6).
constexpr int64_t sum_part(int cg, int64_t T) { return cg == 2 ? 512 : T <= 2 ? 128 : 256; }

// What the epilogue does with the accumulator.
enum : int { kEpiSoftmax = 0, kEpiLogitGrad = 1, kEpiProduct = 2 };

// Offsets behind the stages: staging chunks, then barriers.
constexpr int kHeadStageBytes = kHeadWarps<2, kBackward> * kEpiBufBytes;
constexpr int kHeadBars = 2 * kHeadMaxStages + 4 + 2 + 8;
constexpr int kHeadShares = 3 * 128 * 8;  // forward: partial softmaxes of up to three quarters of a tile's columns for each of its rows
constexpr int kHeadTail = kHeadBars * 8 + 16;

// Division of n < 2^31 by a number that the host knows: with 2^shift < d <=
// 2^(shift + 1) and m = ceil(2^(32 + shift) / d), n m / 2^(32 + shift) is above
// n / d by less than 2^-(shift + 1) <= 1 / d. Short units would otherwise wait
// for the divisions of their places.
struct Divisor {
    unsigned d, m;
    int shift;
    __host__ __device__ __forceinline__ int operator()(int n) const
    {
        return d == 1 ? n : static_cast<int>(static_cast<unsigned>(static_cast<unsigned long long>(static_cast<unsigned>(n)) * m >> 32) >> shift);
    }
};

// One product of a launch. Its units are tiles (in rasters of group_m tile
// rows), one split of K after another.
struct HeadJob {
    int M, N, K;  // rows, columns, length of the sums
    int tiles_m, tiles_n, units, group_m;
    Divisor by_tiles, by_group, by_rows, by_last_rows;  // tiles, tiles of a raster group, its rows, those of the last group
    int kb_all, kb_unit;  // K blocks of the whole product and of a unit
    int kb_part;          // those that the tensor cores sum before the epilogue takes the sum (a unit's, or fewer)
    int bn, bn_last;      // columns of a tile, and of the last one of a row of tiles
    int a_mn, b_mn;
    int epi;
    // the units are dealt out in turn to all clusters, but for the first
    // `extra` rounds, which go to the clusters from `behind` on: those that have
    // one unit less of the job before
    int behind, extra;
    int v0;  // first column of the piece of the vocabulary
    // products
    int out_type;
    int scaled;              // multiply by scale[1]
    int whole;               // columns that TMA stores, in whole 16-byte words; those behind are stored singly
    void *d;
    long long ldd;
    long long slot_rows;     // rows of the output from one split of K to the next
    const float *c_raw;      // fp32 to add before the scale, rows of ld_raw, or null
    long long ld_raw;
    const void *c_typed;     // values of the output's type to add after it, or null
    long long ld_typed;
};

constexpr int kMaxJobs = 3;

struct HeadMaps {
    CUtensorMap a[kMaxJobs], b[kMaxJobs], d[kMaxJobs];
};

struct HeadParams {
    HeadJob jobs[kMaxJobs];
    int num_jobs;
    int a_rows, b_rows;  // rows of the operands' places in a stage
    int in_bf16, stages;
    unsigned long long timeout_ns;
    int inject;
    unsigned int *status;
    // softmax and its gradient
    const int *targets;
    int T, V;
    float2 *partials;  // [tiles_n][T]: reference and sum, base 2
    float *picked;     // the targets' logits
    const float *lse, *dlosses, *dlse;
    float *scale;      // {what dl is multiplied by, its inverse}
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs of fp32 numbers, worked on by one instruction.
__device__ __forceinline__ uint64_t pair_of(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float2 pair_to(uint64_t p)
{
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
    return v;
}

__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Elements of K in a stage.
template <int CG>
constexpr int kHeadBK = CG == 2 ? 128 : 64;

struct HeadUnit {
    int job;
    int m_blk, n_blk, split, kb0, kb1;
};

// A cluster's units, job after job: every role of both CTAs walks the same, and
// so does the host's listing of them.
struct HeadUnits {
    const HeadJob *jobs;
    int num_jobs, c, G;
    int job = 0, round = 0;

    __device__ __forceinline__ HeadUnits(const HeadParams &p, int cluster, int clusters) : HeadUnits(p.jobs, p.num_jobs, cluster, clusters) {}
    __host__ __device__ __forceinline__ HeadUnits(const HeadJob *js, int n, int cluster, int clusters) : jobs(js), num_jobs(n), c(cluster), G(clusters) {}

    __host__ __device__ __forceinline__ bool next(HeadUnit &h)
    {
        while (job < num_jobs) {
            const HeadJob &j = jobs[job];
            const int late = G - j.behind;  // clusters that are behind
            int u = -1;
            if (round < j.extra) {
                if (c >= j.behind)
                    u = round * late + c - j.behind;
                else
                    round = j.extra;
            }
            if (u < 0)
                u = j.extra * late + (round - j.extra) * G + c;
            ++round;
            if (u >= j.units) {
                if (round <= j.extra) {
                    round = j.extra;
                    continue;
                }
                ++job;
                round = 0;
                continue;
            }
            h.job = job;
            h.split = j.by_tiles(u);
            const int local = u - h.split * static_cast<int>(j.by_tiles.d);
            const int g = j.by_group(local), r = local - g * static_cast<int>(j.by_group.d);
            const int left = j.tiles_m - g * j.group_m;
            const Divisor &rows = left < j.group_m ? j.by_last_rows : j.by_rows;
            h.n_blk = rows(r);
            h.m_blk = g * j.group_m + r - h.n_blk * static_cast<int>(rows.d);
            h.kb0 = h.split * j.kb_unit;
            h.kb1 = j.kb_all < h.kb0 + j.kb_unit ? j.kb_all : h.kb0 + j.kb_unit;
            return true;
        }
        return false;
    }
};

template <int CG>
__device__ ProducerTail head_producer(const HeadParams &p, const HeadMaps &maps, uint32_t smem, uint32_t bar_full, uint32_t bar_empty,
                                      uint32_t bar_inject, uint32_t rank, const Waiter &w)
{
    constexpr int BK = kHeadBK<CG>;
    if (p.inject == kRoleProducer) {
        w.wait(bar_inject, 0u, kRoleProducer | kWaitInjected);
        return ProducerTail{0, 0, 0u};
    }
    const int stages = p.stages, a_rows = p.a_rows;
    const uint32_t a_bytes = static_cast<uint32_t>(a_rows) * BK * 2, stage_bytes = a_bytes + static_cast<uint32_t>(p.b_rows) * BK * 2;
    const uint32_t full_target = CG == 2 ? mapa_shared(bar_full, 0) : bar_full;
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    HeadUnits units(p, blockIdx.x / CG, gridDim.x / CG);
    HeadUnit h;
    const CUtensorMap *map_a = nullptr, *map_b = nullptr;
    OperandBoxes box_a = {}, box_b = {};
    int last_job = -1;
    while (units.next(h)) {
        if (h.job != last_job) {
            const HeadJob &j = p.jobs[h.job];
            last_job = h.job;
            map_a = &maps.a[h.job];
            map_b = &maps.b[h.job];
            box_a = operand_boxes(j.a_mn, 3, a_rows, BK, 2);
        }
        const HeadJob &j = p.jobs[h.job];
        const int b_cols = (h.n_blk == j.tiles_n - 1 ? j.bn_last : j.bn) / CG;
        box_b = operand_boxes(j.b_mn, 3, b_cols, BK, 2);
        const uint32_t tx = CG * (a_bytes + static_cast<uint32_t>(b_cols) * BK * 2);
        const int nbox = max(box_a.nbox, box_b.nbox);
        const int m0 = (h.m_blk * CG + static_cast<int>(rank)) * 128;
        const int n0 = h.n_blk * j.bn + b_cols * static_cast<int>(rank);
        for (int kb = h.kb0; kb < h.kb1; ++kb) {
            if (!w.wait(bar_empty + 8 * stage, phase ^ 1u, kRoleProducer | kWaitEmpty, rank != 0))
                return ProducerTail{min(issued, stages), stage, phase};
            if (rank == 0)
                mbar_arrive_expect_tx(bar_full + 8 * stage, tx);
            const uint32_t sa = smem + static_cast<uint32_t>(stage) * stage_bytes;
            const uint32_t fb = full_target + 8 * stage;
            for (int b = 0; b < nbox; ++b) {
                if (b < box_a.nbox)
                    issue_box<CG>(map_a, sa, fb, box_a, b, m0, kb * BK);
                if (b < box_b.nbox)
                    issue_box<CG>(map_b, sa + a_bytes, fb, box_b, b, n0, kb * BK);
            }
            ++issued;
            if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    return ProducerTail{min(issued, stages), stage, phase};
}

template <int CG>
__device__ void head_mma(const HeadParams &p, uint32_t smem, uint32_t bar_full, uint32_t bar_empty, uint32_t bar_acc_full,
                         uint32_t bar_acc_empty, uint32_t bar_inject, uint32_t tmem, const Waiter &w)
{
    constexpr int BK = kHeadBK<CG>, SLICES = BK / 16;
    if (p.inject == kRoleMma) {
        w.wait(bar_inject, 0u, kRoleMma | kWaitInjected);
        return;
    }
    const int stages = p.stages, a_rows = p.a_rows;
    const uint32_t a_bytes = static_cast<uint32_t>(a_rows) * BK * 2, stage_bytes = a_bytes + static_cast<uint32_t>(p.b_rows) * BK * 2;
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    HeadUnits units(p, blockIdx.x / CG, gridDim.x / CG);
    HeadUnit h;
    int last_job = -1, kb_part = 1;
    uint32_t idesc_all = 0, idesc_last = 0, a_off[SLICES], b_off[SLICES];
    int n_last = 0;
    uint64_t a_desc0 = 0, b_desc0 = 0;
    while (units.next(h)) {
        if (h.job != last_job) {
            const HeadJob &j = p.jobs[h.job];
            const int b_cols = j.bn / CG;
            last_job = h.job;
            kb_part = j.kb_part;
            n_last = j.tiles_n - 1;
            idesc_all = make_idesc_f16(128 * CG, j.bn, p.in_bf16, j.a_mn, j.b_mn);
            idesc_last = make_idesc_f16(128 * CG, j.bn_last, p.in_bf16, j.a_mn, j.b_mn);
            const OperandPacking pa = operand_packing(j.a_mn, 3, a_rows, BK), pb = operand_packing(j.b_mn, 3, b_cols, BK);
            a_desc0 = make_smem_desc(smem, pa.lbo, pa.sbo, pa.swz);
            b_desc0 = make_smem_desc(smem + a_bytes, pb.lbo, pb.sbo, pb.swz);
#pragma unroll
            for (int i = 0; i < SLICES; ++i) {
                a_off[i] = slice_byte_offset(j.a_mn, 3, a_rows, i) >> 4;
                b_off[i] = slice_byte_offset(j.b_mn, 3, b_cols, i) >> 4;
            }
        }
        const uint32_t idesc = h.n_blk == n_last ? idesc_last : idesc_all;
        for (int part = h.kb0; part < h.kb1; part += kb_part) {
            if (!w.wait(bar_acc_empty + 8 * acc, acc_phase ^ 1u, kRoleMma | kWaitAccEmpty, CG == 2))
                return;
            tc_fence_after_sync();
            const uint32_t d = tmem + static_cast<uint32_t>(acc * kAccStride);
            const int end = min(part + kb_part, h.kb1);
            for (int kb = part; kb < end; ++kb) {
                if (!mbar_try_wait(bar_full + 8 * stage, phase) && !w.wait(bar_full + 8 * stage, phase, kRoleMma | kWaitFull))
                    return;
                tc_fence_after_sync();
                const uint64_t at = (static_cast<uint32_t>(stage) * stage_bytes) >> 4;
#pragma unroll
                for (int i = 0; i < SLICES; ++i)
                    mma_f16<CG>(d, a_desc0 + at + a_off[i], b_desc0 + at + b_off[i], idesc, ((kb - part) | i) != 0);
                if constexpr (CG == 2)
                    mma_commit_pair_multicast(bar_empty + 8 * stage);
                else
                    mma_commit<1>(bar_empty + 8 * stage);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if constexpr (CG == 2)
                mma_commit_pair_multicast(bar_acc_full + 8 * acc);
            else
                mma_commit<1>(bar_acc_full + 8 * acc);
            acc ^= 1;
            acc_phase ^= acc == 0 ? 1u : 0u;
        }
    }
}

// ---------------------------------------------------------------- epilogues

// 32 values of a thread's row from TMEM: there after tmem_ld_wait().
__device__ __forceinline__ void fetch_acc32(uint32_t taddr, float *v)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
                 : "r"(taddr)
                 : "memory");
}

// 16 values of a row from TMEM, added to `v`. By 16 rather than 32: beside the
// 128 sums that a thread keeps it has no registers for more.
__device__ __forceinline__ void add_acc16(uint32_t taddr, float *v)
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] += __uint_as_float(r[i]);
}

// One pass over a row's columns with the running reference r (the largest
// value so far, times log2 e, rounded) and s = sum of 2^(l log2 e - r): every
// term takes the same r, so its rounding cancels in r + log2 s. A row that
// holds +inf takes r = 0, so that s is +inf; NaN stays in s.
struct RunningSoftmax {
    float r = -INFINITY, s = 0.0f;

    // All of a thread's values of a tile, the first that it sees.
    template <int N>
    __device__ __forceinline__ void take(const float (&v)[N][32])
    {
        float m[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m[i] = fmaxf(v[0][i], v[1][i]);
#pragma unroll
        for (int i = 8; i < 16 * N; ++i)
            m[i & 7] = fmaxf(m[i & 7], fmaxf(v[i / 32 * 2][i & 31], v[i / 32 * 2 + 1][i & 31]));
        const float top = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), fmaxf(fmaxf(m[4], m[5]), fmaxf(m[6], m[7]))) * kLog2e;
        const float ref = fabsf(top) < INFINITY ? top : 0.0f;
        // a tree of sums, so that a term passes seven additions at most, and small ones
        // gather before they meet a large one: level l waits for its other half
        const uint64_t by = pair_of(kLog2e, kLog2e), less = pair_of(-ref, -ref);
        uint64_t level[5];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            uint64_t e[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float2 l = pair_to(fma_pair(pair_of(v[k][2 * i], v[k][2 * i + 1]), by, less));
                e[k] = pair_of(ex2(l.x), ex2(l.y));
            }
            uint64_t sum = add_pair(e[0], e[1]);
            if constexpr (N == 4)
                sum = add_pair(sum, add_pair(e[2], e[3]));
#pragma unroll
            for (int l = 0; l < 4; ++l)
                if (((i + 1) & ((2 << l) - 1)) == 0)
                    sum = add_pair(level[l], sum);
#pragma unroll
            for (int l = 0; l < 5; ++l)
                if (((i + 1) & ((2 << l) - 1)) == (1 << l))
                    level[l] = sum;
        }
        const float2 u = pair_to(level[4]);
        s = u.x + u.y;
        r = top == INFINITY ? 0.0f : fmaxf(top, -INFINITY);  // NaN, of a row of nothing else, to -inf
    }

    // Another part of the row. A sum of 0 or infinity stays what it is whatever
    // its reference.
    __device__ __forceinline__ void join(float2 o)
    {
        const float top = fmaxf(r, o.x);
        const float ref = top == -INFINITY ? 0.0f : top;
        const float a = r == ref || s == 0.0f || s == INFINITY ? s : s * ex2(r - ref);
        const float b = o.x == ref || o.y == 0.0f || o.y == INFINITY ? o.y : o.y * ex2(o.x - ref);
        r = top;
        s = a + b;
    }
};

// The value of `v` at place `at`, where that is one of its 32.
__device__ __forceinline__ float pick32(const float (&v)[32], int at)
{
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        x = i == at ? v[i] : x;
    return x;
}

// What a row's dl needs: exp2(l log2 e - lse2) * a - [target] * b.
struct RowGrad {
    float lse2 = 0.0f, a = 0.0f, b = 0.0f;
    int target = -1;  // relative to the piece
    bool live = false;
};

// A row's values as they come from memory: asked for a unit ahead, since an
// epilogue that is behind has nothing to wait with.
struct RowValues {
    int y;
    float lse, d, z, by;

    __device__ __forceinline__ void load(const HeadParams &p, int row)
    {
        const int at = min(row, p.T - 1);
        y = __ldcg(p.targets + at);
        lse = __ldcg(p.lse + at);
        d = __ldcg(p.dlosses + at);
        z = p.dlse ? __ldcg(p.dlse + at) : 0.0f;
        by = __ldcg(p.scale);
    }
};

__device__ __forceinline__ RowGrad row_grad(const HeadParams &p, const RowValues &r, int v0)
{
    RowGrad g;
    g.live = static_cast<unsigned>(r.y) < static_cast<unsigned>(p.V);
    if (g.live) {
        g.a = (r.d + r.z) * r.by;
        g.b = r.d * r.by;
        g.lse2 = r.lse * kLog2e;
        g.target = r.y - v0;
    }
    return g;
}

// Store of a staging chunk (128 bytes x 32 rows of one split's output); what lies outside is dropped.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// N elements of a row from column `col` on, zeros past column `cols`; whole
// 16-byte words where all are there. Past L1, as they are read once.
template <typename T, int N>
__device__ __forceinline__ void load_row(const T *row, int col, int cols, bool have, uint32_t (&o)[N * sizeof(T) / 4])
{
    constexpr int WORDS = N * sizeof(T) / 4;
#pragma unroll
    for (int i = 0; i < WORDS; ++i)
        o[i] = 0u;
    if (!have)
        return;
    if (col + N <= cols) {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) {
            const uint4 x = __ldcg(reinterpret_cast<const uint4 *>(row + col) + i);
            o[4 * i] = x.x;
            o[4 * i + 1] = x.y;
            o[4 * i + 2] = x.z;
            o[4 * i + 3] = x.w;
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (col + i < cols)
                o[i] = __ldcg(reinterpret_cast<const unsigned int *>(row) + col + i);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (col + i < cols)
                o[i / 2] |= static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned short *>(row) + col + i)) << (16 * (i & 1));
    }
}

// 64 (16-bit) or 32 (fp32) values of a thread's row into its warp's staging
// chunk (SW128 rows) and on to global memory by TMA (32-byte stores from
// registers: 1 x 131072 x 4096 backward 680 us instead of 600). A TMA store
// writes whole 16-byte words, also the one in which a row ends, so that the map ends before
// it and store_tail writes the rest.
template <int CW>
__device__ __forceinline__ void stage_and_store(const uint32_t (&o)[32], uint32_t sbuf, int lane, const CUtensorMap *tmD, int col, int row,
                                                int split)
{
    if (lane == 0)
        bulk_wait_group_read<0>();  // the chunk's last store has read it
    __syncwarp();
    const uint32_t at = sbuf + static_cast<uint32_t>(lane) * 128u, key = static_cast<uint32_t>(lane) & 7u;
#pragma unroll
    for (int u = 0; u < 8; ++u)
        st_shared_v4(at + ((static_cast<uint32_t>(u) ^ key) << 4), o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        tma_store_3d(tmD, sbuf, col, row, split);
        bulk_commit_group();
    }
}

// Columns lo .. hi - 1 of a chunk that starts at `col`.
template <int CW>
__device__ __forceinline__ void store_tail(const uint32_t (&o)[32], void *row, int col, int lo, int hi)
{
#pragma unroll
    for (int i = 0; i < CW; ++i) {
        if (col + i >= lo && col + i < hi) {
            if constexpr (CW == 32)
                static_cast<uint32_t *>(row)[col + i] = o[i];
            else
                static_cast<uint16_t *>(row)[col + i] = static_cast<uint16_t>(o[i / 2] >> (16 * (i & 1)));
        }
    }
}

// Columns 32 i .. +31 of a chunk in the output's type.
template <int CW>
__device__ __forceinline__ void pack32(const float (&v)[32], int i, int out_type, uint32_t (&o)[32])
{
    if constexpr (CW == 32) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
            o[k] = __float_as_uint(v[k]);
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint32_t four[4];
            pack_out(v + 8 * u, out_type, four);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[16 * i + 4 * u + k] = four[k];
        }
    }
}

// Arrive on the even CTA's barrier for an accumulator this warp has read. The
// reads of TMEM have completed (tcgen05.wait::ld), and nothing that the warp has
// stored is the MMA's to read, so that the release is confined to this CTA's
// shared memory: one of all memory waits for the stores to global memory that
// are on their way (forward 8192 x 32768 x 256 151 us, 7252 x 118755 x 128 441;
// confined 112 and 346).
__device__ __forceinline__ void mbar_arrive_read(uint32_t cluster_bar)
{
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;\n\t"
                 "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
                 : "memory");
}

// An epilogue warp's view of the accumulators: waits for the next one and hands
// it back. Warp w has TMEM lanes 32 (w mod 4) .. +31 and a half or a quarter of the
// columns.
template <int CG>
struct Accumulators {
    uint32_t bar_full, bar_empty, tmem;  // bar_empty: the even CTA's
    int acc = 0;
    uint32_t phase = 0;

    __device__ __forceinline__ bool take(const Waiter &w, uint32_t rank)
    {
        const bool ok = w.wait(bar_full + 8 * acc, phase, kRoleEpilogue | kWaitAccFull, rank != 0);
        tc_fence_after_sync();
        return __all_sync(0xffffffffu, ok) != 0;
    }

    __device__ __forceinline__ void release(int lane)
    {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
            if constexpr (CG == 2)
                mbar_arrive_read(bar_empty + 8 * acc);
            else
                mbar_arrive(bar_empty + 8 * acc);
        }
        acc ^= 1;
        phase ^= acc == 0 ? 1u : 0u;
    }

    __device__ __forceinline__ uint32_t columns(int q, int c) const
    {
        return tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(acc * kAccStride + c);
    }
};

// Forward: each tile's partial softmax. The warps that share a row join
// theirs through shared memory.
template <int CG>
__device__ void softmax_epilogue(const HeadParams &p, float2 *shares, uint32_t bar_shares, Accumulators<CG> a, uint32_t rank, int warp, int lane,
                                 const Waiter &w)
{
    constexpr int SHARES = kHeadWarps<CG, kForward> / 4, N = 8 / SHARES;  // warps of a row, their chunks of 32 columns
    const int q = warp & 3, share = (warp - 2) >> 2;
    float2 *const slot = shares + 32 * q + lane;  // 128 from one share's to the next
    const uint32_t bar_ready = bar_shares + 16 * q, bar_free = bar_ready + 8;
    uint32_t phase = 0;
    HeadUnits units(p, blockIdx.x / CG, gridDim.x / CG);
    const HeadJob &j = p.jobs[0];
    HeadUnit h;
    while (units.next(h)) {
        const int m0 = (h.m_blk * CG + static_cast<int>(rank)) * 128 + 32 * q, row = m0 + lane;
        const int n0 = h.n_blk * j.bn, cols = min(j.bn, j.N - n0);
        const int y = row < p.T ? __ldcg(p.targets + row) - n0 : -1;
        const bool rows = m0 < p.T;  // the same for all warps of the row
        // the parts of the sums over K, added up in registers with fp32 rounding
        float v[N][32];
        for (int part = 0; part < j.kb_all; part += j.kb_part) {
            if (!a.take(w, rank))
                return;
            if (part == 0) {
                // all of them: columns past the tile's lie in TMEM too, and are masked below
#pragma unroll
                for (int i = 0; i < N; ++i)
                    fetch_acc32(a.columns(q, 32 * (share + SHARES * i)), v[i]);
                tmem_ld_wait();
            } else if (rows) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int c = 32 * (share + SHARES * i);
                    if (c < cols) {
                        add_acc16(a.columns(q, c), v[i]);
                        add_acc16(a.columns(q, c + 16), v[i] + 16);
                    }
                }
            }
            a.release(lane);
        }
        if (!rows)
            continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = 32 * (share + SHARES * i);
            if (c + 32 > cols) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    v[i][k] = c + k < cols ? v[i][k] : -INFINITY;
            }
        }
        RunningSoftmax sm;
        sm.take(v);
        // the target comes last: it has been on its way from memory meanwhile
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = 32 * (share + SHARES * i);
            const bool mine = y >= c && y < min(c + 32, cols);
            if (__any_sync(0xffffffffu, mine)) {
                const float x = pick32(v[i], y - c);
                if (mine)
                    p.picked[row] = x;
            }
        }
        if (share > 0) {
            if (!__all_sync(0xffffffffu, w.wait(bar_free, phase ^ 1u, kRoleEpilogue | kWaitPartial)))
                return;
            slot[128 * (share - 1)] = make_float2(sm.r, sm.s);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_ready);
        } else {
            if (!__all_sync(0xffffffffu, w.wait(bar_ready, phase, kRoleEpilogue | kWaitPartial)))
                return;
#pragma unroll
            for (int i = 0; i < SHARES - 1; ++i)
                sm.join(slot[128 * i]);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_free);
            if (row < p.T)
                p.partials[static_cast<long long>(h.n_blk) * p.T + row] = make_float2(sm.r, sm.s);
        }
        phase ^= 1u;
    }
}

// 64 columns of a tile of dl, from column c on.
__device__ __forceinline__ void logit_grad_chunk(const HeadParams &p, const CUtensorMap *map, const RowGrad &g, float (&lo)[32], float (&hi)[32],
                                                 int m0, int n0, int c, uint32_t sbuf, int lane)
{
    const uint64_t by = pair_of(kLog2e, kLog2e), less = pair_of(-g.lse2, -g.lse2), scale = pair_of(g.a, g.a);
    uint32_t o[32];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float (&v)[32] = i == 0 ? lo : hi;
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            const float2 l = pair_to(fma_pair(pair_of(v[k], v[k + 1]), by, less));
            const float2 d = pair_to(mul_pair(pair_of(ex2(l.x), ex2(l.y)), scale));
            v[k] = d.x;
            v[k + 1] = d.y;
        }
        const int at = g.target - (n0 + c + 32 * i);
        if (__any_sync(0xffffffffu, at >= 0 && at < 32)) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
                v[k] -= at == k ? g.b : 0.0f;
        }
        pack32<64>(v, i, p.in_bf16 ? 1 : 2, o);
    }
#pragma unroll
    for (int k = 0; k < 32; ++k)
        o[k] = g.live ? o[k] : 0u;  // whatever the row of a token without a loss made of them
    stage_and_store<64>(o, sbuf, lane, map, n0 + c, m0, 0);
}

// One tile of dl whose sums over K are one part: each 64 columns as they come.
template <int CG>
__device__ __forceinline__ void logit_grad_tile(const HeadParams &p, const CUtensorMap *map, const RowGrad &g, const Accumulators<CG> &a, int q,
                                                int half, int m0, int n0, int cols, uint32_t sbuf, int lane)
{
    for (int c = 64 * half; c < cols; c += 128) {
        float x[2][32];
        fetch_acc32(a.columns(q, c), x[0]);
        fetch_acc32(a.columns(q, c + 32), x[1]);
        tmem_ld_wait();
        logit_grad_chunk(p, map, g, x[0], x[1], m0, n0, c, sbuf, lane);
    }
}

// One tile of dl from the parts of its sums over K, added up in registers as the
// forward pass adds them. False if a wait has run out.
template <int CG>
__device__ __forceinline__ bool logit_grad_parts(const HeadParams &p, const HeadJob &j, const CUtensorMap *map, Accumulators<CG> &a, int q,
                                                 int half, int m0, int n0, int cols, uint32_t sbuf, int lane, uint32_t rank, const Waiter &w)
{
    const bool rows = m0 < j.M;  // the same for the whole warp
    auto column = [&](int i) { return 64 * half + 128 * (i >> 1) + 32 * (i & 1); };
    float v[4][32] = {};
    RowValues values = {};
    for (int part = 0; part < j.kb_all; part += j.kb_part) {
        if (part + j.kb_part >= j.kb_all)
            values.load(p, m0 + lane);  // on their way while the last part is waited for
        if (!a.take(w, rank))
            return false;
        if (rows) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = column(i);
                if (c < cols) {
                    add_acc16(a.columns(q, c), v[i]);
                    add_acc16(a.columns(q, c + 16), v[i] + 16);
                }
            }
        }
        a.release(lane);
    }
    if (rows) {
        const RowGrad g = row_grad(p, values, j.v0);
#pragma unroll
        for (int i = 0; i < 4; i += 2)
            if (column(i) < cols)
                logit_grad_chunk(p, map, g, v[i], v[i + 1], m0, n0, column(i), sbuf, lane);
    }
    return true;
}

// One tile of a gradient, in chunks of 32 (fp32) or 64 columns.
template <int CG, int CW>
__device__ __forceinline__ void product_tile(const HeadParams &p, const HeadJob &j, const CUtensorMap *map, const Accumulators<CG> &a, int q,
                                             int half, int m0, int n0, int cols, int split, uint32_t sbuf, int lane)
{
    const int row = m0 + lane;
    const bool have = row < j.M;
    const float by = j.scaled ? __ldcg(p.scale + 1) : 1.0f;
    for (int c = CW * half; c < cols; c += 2 * CW) {
        uint32_t o[32];
        const int col = n0 + c;
#pragma unroll
        for (int i = 0; i < CW / 32; ++i) {
            float v[32];
            uint32_t old[32];
            const int at = col + 32 * i;
            if (j.c_raw)
                load_row<float, 32>(j.c_raw + (split * j.slot_rows + row) * j.ld_raw, at, j.N, have, old);
            __syncwarp();
            fetch_acc32(a.columns(q, c + 32 * i), v);
            tmem_ld_wait();
            if (j.c_raw) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    v[k] += __uint_as_float(old[k]);
            }
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
                const float2 d = pair_to(mul_pair(pair_of(v[k], v[k + 1]), pair_of(by, by)));
                v[k] = d.x;
                v[k + 1] = d.y;
            }
            if (j.c_typed) {
                if constexpr (CW == 32) {
                    load_row<float, 32>(static_cast<const float *>(j.c_typed) + row * j.ld_typed, at, j.N, have, old);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        v[k] += __uint_as_float(old[k]);
                } else {
                    uint32_t two[16];
                    load_row<__half, 32>(static_cast<const __half *>(j.c_typed) + row * j.ld_typed, at, j.N, have, two);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t four[4] = {two[4 * u], two[4 * u + 1], two[4 * u + 2], two[4 * u + 3]};
                        float f[8];
                        unpack_in(four, j.out_type, f);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            v[8 * u + k] += f[k];
                    }
                }
            }
            pack32<CW>(v, i, j.out_type, o);
        }
        if (col < j.whole)
            stage_and_store<CW>(o, sbuf, lane, map, col, m0, split);
        if (col + CW > j.whole && j.whole < j.N && have)
            store_tail<CW>(o, static_cast<char *>(j.d) + row * j.ldd * (CW == 32 ? 4 : 2), col, j.whole, j.N);
    }
}

// Backward: tiles of dl, dX and dW.
template <int CG, int MODE>
__device__ void gradient_epilogue(const HeadParams &p, const HeadMaps &maps, uint32_t sbuf, Accumulators<CG> a, uint32_t rank, int warp,
                                  int lane, const Waiter &w)
{
    constexpr bool PARTS = MODE == kBackwardParts;
    const int q = warp & 3, half = (warp - kHeadFirstWarp<MODE>) >> 2;
    HeadUnits units(p, blockIdx.x / CG, gridDim.x / CG);
    auto first_row = [&](const HeadUnit &u) { return (u.m_blk * CG + static_cast<int>(rank)) * 128 + 32 * q; };
    HeadUnit h;
    RowValues values = {}, next_values = {};
    bool more = units.next(h);
    if (!PARTS && more && p.jobs[h.job].epi == kEpiLogitGrad)
        next_values.load(p, first_row(h) + lane);
    while (more) {
        const HeadJob &j = p.jobs[h.job];
        const CUtensorMap *const map = &maps.d[h.job];
        const int m0 = first_row(h), split = h.split;
        const int n0 = h.n_blk * j.bn, cols = min(j.bn, j.N - n0);
        values = next_values;
        more = units.next(h);
        if (!PARTS && more && p.jobs[h.job].epi == kEpiLogitGrad)
            next_values.load(p, first_row(h) + lane);
        if (PARTS && j.epi == kEpiLogitGrad) {
            if (!logit_grad_parts<CG>(p, j, map, a, q, half, m0, n0, cols, sbuf, lane, rank, w))
                return;
            continue;
        }
        if (!a.take(w, rank))
            return;
        if (m0 < j.M) {  // the same for the whole warp
            if (!PARTS && j.epi == kEpiLogitGrad)
                logit_grad_tile<CG>(p, map, row_grad(p, values, j.v0), a, q, half, m0, n0, cols, sbuf, lane);
            else if (j.out_type == 0)
                product_tile<CG, 32>(p, j, map, a, q, half, m0, n0, cols, split, sbuf, lane);
            else
                product_tile<CG, 64>(p, j, map, a, q, half, m0, n0, cols, split, sbuf, lane);
        }
        a.release(lane);
    }
}

// ---------------------------------------------------------------- kernel

template <int CG, int MODE>
__global__ void __launch_bounds__(kHeadThreads<CG, MODE>, 1) head_kernel(const __grid_constant__ HeadMaps maps, const __grid_constant__ HeadParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    const uint32_t rank = CG == 2 ? cluster_ctarank() & 1u : 0u;
    const int stages = p.stages;
    const uint32_t staging = base + static_cast<uint32_t>(stages) * static_cast<uint32_t>(p.a_rows + p.b_rows) * kHeadBK<CG> * 2;
    const uint32_t bars = staging + (MODE == kForward ? kHeadShares : kHeadStageBytes);
    const uint32_t bar_full = bars, bar_empty = bar_full + 8 * kHeadMaxStages;
    const uint32_t bar_acc_full = bar_empty + 8 * kHeadMaxStages, bar_acc_empty = bar_acc_full + 16;
    const uint32_t bar_drain = bar_acc_empty + 16, bar_inject = bar_drain + 8;
    const uint32_t bar_shares = bar_inject + 8, misc = bar_shares + 64;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + (misc - base));
    volatile uint32_t *abort_flag = tmem_slot + 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_acc_full + 8 * b, 1);
            mbar_init(bar_acc_empty + 8 * b, kHeadWarps<CG, MODE> * CG);
        }
        mbar_init(bar_drain, 1);
        mbar_init(bar_inject, 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar_shares + 16 * i, kHeadWarps<CG, MODE> / 4 - 1);
            mbar_init(bar_shares + 16 * i + 8, 1);
        }
        *abort_flag = 0u;
        fence_mbar_init();
        for (int j = 0; j < p.num_jobs; ++j) {
            prefetch_tensormap(&maps.a[j]);
            prefetch_tensormap(&maps.b[j]);
            if constexpr (MODE != kForward)
                prefetch_tensormap(&maps.d[j]);
        }
    }
    if (warp == 1) {
        tmem_alloc<CG>(smem_u32(tmem_slot), 2 * kAccStride);
        tmem_relinquish<CG>();
    }
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (CG == 2)
        cluster_sync_all();  // the peer's barriers exist before anything signals them
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_start();

    Waiter w;
    w.timeout_ns = p.timeout_ns;
    w.abort_flag = abort_flag;
    w.status = p.status;
    w.all_cluster_scope = false;
    ProducerTail tail{0, 0, 0u};
    if (warp < kHeadFirstWarp<MODE>) {
        if constexpr (MODE == kBackwardParts)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kBackIssueRegs));
        if (warp == 0 && lane == 0) {
            // what kernels before this one wrote by ordinary stores is read by TMA
            asm volatile("fence.proxy.async;" ::: "memory");
            tail = head_producer<CG>(p, maps, base, bar_full, bar_empty, bar_inject, rank, w);
        } else if (warp == 1 && lane == 0 && rank == 0) {
            head_mma<CG>(p, base, bar_full, bar_empty, bar_acc_full, bar_acc_empty, bar_inject, tmem, w);
            mma_commit<CG>(bar_drain);
            w.drain(bar_drain, 0u, 100000000ull);
        }
    } else {
        if constexpr (MODE == kBackwardParts)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kBackEpiRegs));
        const Accumulators<CG> a{bar_acc_full, CG == 2 ? mapa_shared(bar_acc_empty, 0) : bar_acc_empty, tmem};
        if constexpr (MODE == kForward)
            softmax_epilogue<CG>(p, reinterpret_cast<float2 *>(smem + (staging - base)), bar_shares, a, rank, warp, lane, w);
        else
            gradient_epilogue<CG, MODE>(p, maps, staging + static_cast<uint32_t>((warp - kHeadFirstWarp<MODE>) * kEpiBufBytes), a, rank, warp, lane, w);
        if (MODE != kForward && lane == 0)
            bulk_wait_group<0>();  // stores have finished reading shared memory
    }
    __syncwarp();
    __syncthreads();  // every role has returned: the abort flag is final
    if (*abort_flag) {
        // as in gemm_kernel.cuh: loads still in flight land before the CTA exits
        if (warp == 0 && lane == 0 && rank == 0) {
            for (int i = 1; i <= tail.inflight; ++i) {
                int s = tail.stage - i;
                uint32_t ph = tail.phase;
                if (s < 0) {
                    s += stages;
                    ph ^= 1u;
                }
                w.drain(bar_full + 8 * s, ph, 2000000ull);
            }
        }
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 20000ull)
            __nanosleep(1000);
    }
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (CG == 2)
        cluster_sync_all();  // no CTA exits while the other may still write into it
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc<CG>(tmem, 2 * kAccStride);
    }
}

// ---------------------------------------------------------------- around the products

// The normaliser and loss of each token from its partial softmaxes: a block has
// ROWS tokens (8, or 1 where tokens are few), and 16 warps share the partials, a
// warp 32 / ROWS of them at a time. r
// is a maximum over the partials, so that the sum is in range; the loss is taken
// in base 2, where the target's logit cancels against r before anything is
// rounded.
constexpr int kCombineWarps = 16;

template <int ROWS>
__global__ void __launch_bounds__(32 * kCombineWarps)
    head_combine_kernel(const float2 *partials, int parts, long long T, const int *targets, int V, float *losses, float *lse)
{
    __shared__ float2 part[kCombineWarps][ROWS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int SHARES = 32 / ROWS, step = SHARES * kCombineWarps;
    const long long row = static_cast<long long>(blockIdx.x) * ROWS + lane % ROWS;
    const int first = warp * SHARES + lane / ROWS;
    grid_start();
    RunningSoftmax sm;
    if (row < T) {
        for (int i = first; i < parts; i += 8 * step) {
            float2 o[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                o[u] = i + u * step < parts ? __ldcg(partials + (i + u * step) * T + row) : make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                sm.join(o[u]);
        }
    }
#pragma unroll
    for (int o = 16; o >= ROWS; o >>= 1) {
        float2 other;
        other.x = __shfl_xor_sync(0xffffffffu, sm.r, o);
        other.y = __shfl_xor_sync(0xffffffffu, sm.s, o);
        sm.join(other);
    }
    if (lane < ROWS)
        part[warp][lane] = make_float2(sm.r, sm.s);
    __syncthreads();
    if (warp != 0 || lane >= ROWS || row >= T)
        return;
#pragma unroll
    for (int i = 1; i < kCombineWarps; ++i)
        sm.join(part[i][lane]);
    const int y = __ldcg(targets + row);
    const bool live = static_cast<unsigned>(y) < static_cast<unsigned>(V);
    const float ref = sm.r == -INFINITY ? 0.0f : sm.r;
    const float log2s = log2f(sm.s);
    lse[row] = live ? (ref + log2s) * kLn2 : 0.0f;
    losses[row] = live ? (fmaf(-__ldcg(losses + row), kLog2e, ref) + log2s) * kLn2 : 0.0f;
}

// What the gradients need of all tokens: block 0 finds the largest |dloss| +
// |dlse| of the live ones and sets scale = {c / largest, largest / c}, so that
// dl is at most c in magnitude whatever the caller's scaling (c = 1 for bf16,
// 2^14 for fp16, whose small probabilities would otherwise be subnormal);
// the other blocks copy X with the rows of tokens without a loss zeroed, so
// that what such a row holds (a NaN, say) does not reach dW as 0 * NaN.
constexpr int kPrepareThreads = 512;

__global__ void __launch_bounds__(kPrepareThreads)
    head_prepare_kernel(const uint4 *x, long long ldx16, uint4 *xs, long long ld16, int K, long long T, const int *targets, int V,
                        const float *dlosses, const float *dlse, float c, float *scale)
{
    grid_start();
    if (blockIdx.x == 0) {
        __shared__ float top[kPrepareThreads / 32];
        float m = 0.0f;
#pragma unroll 4
        for (long long t = threadIdx.x; t < T; t += kPrepareThreads) {
            const float d = fabsf(__ldcg(dlosses + t)) + (dlse ? fabsf(__ldcg(dlse + t)) : 0.0f);
            m = fmaxf(m, static_cast<unsigned>(__ldcg(targets + t)) < static_cast<unsigned>(V) ? d : 0.0f);
        }
        m = warp_max(m);
        if ((threadIdx.x & 31) == 0)
            top[threadIdx.x >> 5] = m;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kPrepareThreads / 32; ++i)
                m = fmaxf(m, top[i]);
            m = fminf(fmaxf(m, 1e-30f), 3e38f);
            scale[0] = c / m;
            scale[1] = m / c;
        }
        return;
    }
    if (!xs)
        return;
    const int words = (K + 7) / 8;
    const long long all = T * words, step = (gridDim.x - 1ll) * kPrepareThreads;
    for (long long i = (blockIdx.x - 1ll) * kPrepareThreads + threadIdx.x; i < all; i += step) {
        const long long t = i / words;
        const int k = static_cast<int>(i - t * words);
        const bool live = static_cast<unsigned>(__ldcg(targets + t)) < static_cast<unsigned>(V);
        if (8 * k + 8 <= K) {
            xs[t * ld16 + k] = live ? __ldcg(x + t * ldx16 + k) : make_uint4(0, 0, 0, 0);
        } else {  // nothing past the row's end is read; what is past it in the copy is never used
            const unsigned short *from = reinterpret_cast<const unsigned short *>(x + t * ldx16 + k);
            uint16_t *to = reinterpret_cast<uint16_t *>(xs + t * ld16 + k);
            for (int j = 0; j < K - 8 * k; ++j)
                to[j] = live ? __ldcg(from + j) : static_cast<uint16_t>(0);
        }
    }
}

// dX from the sums over parts of the vocabulary, in a fixed order. GROUPS of a
// block's 256 threads take every so-manieth part of an item, four columns: many
// parts of few items would leave each thread with a long chain of loads (383 x
// 108285 x 178 backward 121 us, 99 by groups of 8).
constexpr int kSumGroups = 8;

template <typename D, int GROUPS>
__global__ void __launch_bounds__(256)
    head_sum_kernel(const float *parts, int n, long long stride, long long ld, long long T, int K, const float *scale, D *d, long long ldd)
{
    constexpr int ITEMS = 256 / GROUPS;
    __shared__ float4 sums[GROUPS > 1 ? GROUPS : 1][ITEMS];
    const int item = static_cast<int>(threadIdx.x) % ITEMS, group = static_cast<int>(threadIdx.x) / ITEMS;
    grid_start();
    const float by = __ldcg(scale + 1);
    const int words = (K + 3) / 4;
    const long long all = T * words, step = static_cast<long long>(gridDim.x) * ITEMS;
    for (long long first = static_cast<long long>(blockIdx.x) * ITEMS; first < all; first += step) {
        const long long i = min(first + item, all - 1);
        const long long t = i / words;
        const int k = 4 * static_cast<int>(i - t * words);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](const float4 &v) {
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        };
#pragma unroll 4
        for (int j = group; j < n; j += GROUPS)
            add(__ldcg(reinterpret_cast<const float4 *>(parts + j * stride + t * ld + k)));
        if constexpr (GROUPS > 1) {
            __syncthreads();  // the sums of the items before have been read
            sums[group][item] = s;
            __syncthreads();
            if (group > 0)
                continue;
#pragma unroll
            for (int j = 1; j < GROUPS; ++j)
                add(sums[j][item]);
        }
        if (first + item >= all)
            continue;
        D *o = d + t * ldd + k;
        const float v[4] = {s.x * by, s.y * by, s.z * by, s.w * by};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (k + j < K)
                o[j] = from_float<D>(v[j]);
    }
}

// Zeros for dW when there is no token.
__global__ void __launch_bounds__(256) head_zero_kernel(uint8_t *d, long long ld_bytes, long long rows, long long row_bytes)
{
    grid_start();
    for (long long r = blockIdx.x; r < rows; r += gridDim.x)
        for (long long i = 2 * static_cast<int>(threadIdx.x); i < row_bytes; i += 512)
            *reinterpret_cast<uint16_t *>(d + r * ld_bytes + i) = 0;
}

// ---------------------------------------------------------------- few tokens, backward

// One or two tokens: one pass over the weights by fp32 arithmetic. A group of
// threads has R words at a time, each thread eight columns of them: their dot
// products with the tokens' rows, summed over the group, give dl, with which
// the same registers make the words' rows of dW and add to dX. Bound by memory,
// which holds the weights once and their gradient once (the tiles of the
// products read the weights twice): 1 x 131072 x 4096 in 375 us, of 322 at the
// copy rate, 2 x 131072 x 4096 in 368, 1 x 32000 x 1024 in 33 (by tiles 607, 610
// and 60). Four tokens, of which registers hold two words at a time, took as
// long as by tiles. (One token's eight words leave some 26 registers of a thread in
// memory, 104 bytes; two tokens' four none.)
constexpr int kFewThreads = 512;  // K <= 8 * 512
constexpr int kFewBlocks = 152;   // one for each SM of the GPU this is built for

struct FewParams {
    const void *x, *w;
    void *dw;
    float *parts;  // [block][T][ld_parts], or null
    long long ldx, ldw, lddw, ld_parts;
    int T, V, K, x_threads, dw_type, accumulate;
    const int *targets;
    const float *lse, *dlosses, *dlse;
};

// Eight 16-bit values as pairs.
template <typename I>
__device__ __forceinline__ void widen(const uint4 &v, uint64_t (&o)[4])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<I, __nv_bfloat16>::value) {
            o[i] = pair_of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            o[i] = pair_of(f.x, f.y);
        }
    }
}

// Eight 16-bit values of a row from column k on, zeros past its end.
__device__ __forceinline__ uint4 load_eight(const uint16_t *row, int k, int K, bool have)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    if (have && k + 8 <= K) {
        v = __ldcg(reinterpret_cast<const uint4 *>(row + k));
    } else if (have && k < K) {
        uint32_t w[4] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < K)
                w[i / 2] |= static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned short *>(row) + k + i)) << (16 * (i & 1));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}

template <typename D>
__device__ __forceinline__ void store_eight(void *row, int k, int K, int accumulate, float (&v)[8])
{
    D *p = static_cast<D *>(row) + k;
    if (k + 8 <= K) {
        float old[8];
        if (accumulate) {
            load8<D, true>(p, 0, 1, 8, old);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += old[i];
        }
        store8<D, true>(p, 0, 1, 8, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < K)
                p[i] = from_float<D>(accumulate ? v[i] + to_float(p[i]) : v[i]);
    }
}

template <typename I, int TT>
__global__ void __launch_bounds__(kFewThreads, 1) head_few_kernel(const FewParams p)
{
    constexpr int R = 8 / TT, N = R * TT;  // words at a time; their dot products
    extern __shared__ float few_smem[];             // [TT][8 * x threads] of dX at the end
    __shared__ float dots[2][kFewThreads / 32][N];
    const int tid = threadIdx.x, group = threadIdx.y, lane = tid & 31, k = 8 * tid;
    const int warps = p.x_threads / 32, warp = tid >> 5;  // of the group
    const int groups = static_cast<int>(blockDim.y);
    grid_start();
    uint64_t x[TT][4], acc[TT][4] = {};
    // lane j has the constants of token j % TT
    const int t_of = lane % TT;
    RowGrad g;
    if (t_of < p.T) {
        const int y = __ldcg(p.targets + t_of);
        g.live = static_cast<unsigned>(y) < static_cast<unsigned>(p.V);
        if (g.live) {
            const float d = __ldcg(p.dlosses + t_of);
            g.a = d + (p.dlse ? __ldcg(p.dlse + t_of) : 0.0f);
            g.b = d;
            g.lse2 = __ldcg(p.lse + t_of) * kLog2e;
            g.target = y;
        }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const bool live = __shfl_sync(0xffffffffu, g.live, t);
        widen<I>(load_eight(static_cast<const uint16_t *>(p.x) + (t < p.T ? t : 0) * p.ldx, k, p.K, live), x[t]);
    }
    const uint16_t *weights = static_cast<const uint16_t *>(p.w);
    const long long step = static_cast<long long>(gridDim.x) * groups * R;
    long long v0 = (static_cast<long long>(blockIdx.x) * groups + group) * R;
    uint4 next[R];  // asked for a step ahead
#pragma unroll
    for (int r = 0; r < R; ++r)
        next[r] = load_eight(weights + (v0 + r) * p.ldw, k, p.K, v0 + r < p.V);
    for (int turn = 0; v0 < p.V; v0 += step, turn ^= 1) {
        uint4 w[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            w[r] = next[r];
            next[r] = load_eight(weights + (v0 + step + r) * p.ldw, k, p.K, v0 + step + r < p.V);
        }
        float dot[N];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint64_t words[4];
            widen<I>(w[r], words);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                uint64_t s = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s = fma_pair(x[t][i], words[i], s);
                const float2 two = pair_to(s);
                dot[r * TT + t] = two.x + two.y;
            }
        }
        // the warp's sums: halves of the values change places until a lane has one
        int at = 0;
#pragma unroll
        for (int m = N / 2, o = 16; o > 0; o >>= 1, m /= 2) {
            if (m > 0) {
                const bool upper = lane & o;
                at += upper ? m : 0;
#pragma unroll
                for (int i = 0; i < m; ++i) {
                    const float send = upper ? dot[i] : dot[i + m];
                    const float keep = upper ? dot[i + m] : dot[i];
                    dot[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
            } else {
                dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], o);
            }
        }
        if (lane % (32 / N) == 0)
            dots[turn][group * warps + warp][at] = dot[0];
        if (warps == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(p.x_threads) : "memory");
        // dl of word (lane % N) / TT and token lane % TT, in every warp
        float l = 0.0f;
        for (int i = lane / N; i < warps; i += 32 / N)
            l += dots[turn][group * warps + i][lane % N];
#pragma unroll
        for (int o = N; o < 32; o <<= 1)
            l += __shfl_xor_sync(0xffffffffu, l, o);
        const long long v = v0 + (lane % N) / TT;
        const float dl = g.live && v < p.V ? ex2(fmaf(l, kLog2e, -g.lse2)) * g.a - (v == g.target ? g.b : 0.0f) : 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint64_t words[4], sums[4] = {};
            widen<I>(w[r], words);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const float d = __shfl_sync(0xffffffffu, dl, r * TT + t);
                const uint64_t two = pair_of(d, d);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sums[i] = fma_pair(two, x[t][i], sums[i]);
                    acc[t][i] = fma_pair(two, words[i], acc[t][i]);
                }
            }
            float out[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 two = pair_to(sums[i]);
                out[2 * i] = two.x;
                out[2 * i + 1] = two.y;
            }
            if (p.dw && v0 + r < p.V && k < p.K) {
                if (p.dw_type == GEMM_OUT_F32)
                    store_eight<float>(static_cast<float *>(p.dw) + (v0 + r) * p.lddw, k, p.K, p.accumulate, out);
                else if (p.dw_type == GEMM_OUT_BF16)
                    store_eight<__nv_bfloat16>(static_cast<__nv_bfloat16 *>(p.dw) + (v0 + r) * p.lddw, k, p.K, p.accumulate, out);
                else
                    store_eight<__half>(static_cast<__half *>(p.dw) + (v0 + r) * p.lddw, k, p.K, p.accumulate, out);
            }
        }
    }
    if (!p.parts)
        return;
    // dX of the block's groups, in their order
    float mine[TT][8];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 two = pair_to(acc[t][j]);
            mine[t][2 * j] = two.x;
            mine[t][2 * j + 1] = two.y;
        }
    for (int i = 0; i < groups; ++i) {
        __syncthreads();
        if (group == i) {
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float *s = few_smem + (t * 8 + j) * p.x_threads + tid;
                    if (i > 0)
                        mine[t][j] += *s;
                    if (i + 1 < groups)
                        *s = mine[t][j];
                }
        }
    }
    if (group == groups - 1 && k < p.K) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int j = 0; j < 8; j += 4)
                if (t < p.T)
                    *reinterpret_cast<float4 *>(p.parts + (static_cast<long long>(blockIdx.x) * p.T + t) * p.ld_parts + k + j) =
                        make_float4(mine[t][j], mine[t][j + 1], mine[t][j + 2], mine[t][j + 3]);
    }
}

// dX from the blocks' parts: eight threads share an element's parts, in a fixed order.
template <typename D>
__global__ void __launch_bounds__(256) head_few_sum_kernel(const float *parts, int n, long long ld, int T, int K, D *d, long long ldd)
{
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int k = static_cast<int>(blockIdx.x) * 32 + lane, t = static_cast<int>(blockIdx.y);
    grid_start();
    float s = 0.0f;
    if (k < K) {
#pragma unroll 8
        for (int i = part; i < n; i += 8)
            s += __ldcg(parts + (static_cast<long long>(i) * T + t) * ld + k);
    }
    sums[part][lane] = s;
    __syncthreads();
    if (part == 0 && k < K) {
#pragma unroll
        for (int i = 1; i < 8; ++i)
            s += sums[i][lane];
        d[t * ldd + k] = from_float<D>(s);
    }
}

// ---------------------------------------------------------------- host

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

gemm_status_t encode_16(CUtensorMap *m, int in_bf16, const void *ptr, int mn_major, int64_t mn, int64_t k, int64_t ld, int rows, int bk)
{
    const CUtensorMapDataType dt = in_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const uint64_t dims[2] = {static_cast<uint64_t>(mn_major ? mn : k), static_cast<uint64_t>(mn_major ? k : mn)};
    const uint64_t strides[1] = {static_cast<uint64_t>(ld) * 2};
    const uint32_t box[2] = {64, static_cast<uint32_t>(mn_major ? bk : rows)};
    return host_encode_tiled(m, dt, 2, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

gemm_status_t encode_out(CUtensorMap *m, int type, const void *ptr, int64_t rows, int64_t cols, int64_t ld, int64_t splits = 1)
{
    const int es = type_bytes(type);
    const CUtensorMapDataType dt = type == GEMM_OUT_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : type == GEMM_OUT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                           : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const uint64_t row = static_cast<uint64_t>(ld) * es;
    // (a map has a column at least: of one without whole words no chunk is stored)
    const uint64_t dims[3] = {static_cast<uint64_t>(std::max<int64_t>(cols, 16 / es)), static_cast<uint64_t>(rows),
                              static_cast<uint64_t>(splits)};
    // one split: its stride is never walked, and may not be one that a tensor map refuses
    const uint64_t strides[2] = {row, splits > 1 ? row * rows : row};
    const uint32_t box[3] = {static_cast<uint32_t>(128 / es), 32, 1};
    return host_encode_tiled(m, dt, 3, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Columns of a caller's row that make up whole 16-byte words.
int64_t whole_words(int64_t cols, int type) { return cols - cols % (16 / type_bytes(type)); }

// One operand of a product.
struct Operand {
    const void *ptr;
    int64_t ld;
};

Divisor divisor(int64_t d)
{
    Divisor v = {static_cast<unsigned>(d), 0u, 0};
    if (d > 1) {
        while ((int64_t(1) << (v.shift + 1)) < d)
            ++v.shift;  // 2^shift < d <= 2^(shift + 1)
        v.m = static_cast<unsigned>(((uint64_t(1) << (32 + v.shift)) + d - 1) / d);
    }
    return v;
}

// A product of a launch as the host builds it.
struct Job {
    HeadJob j;
    CUtensorMap a, b, d;
    int64_t cost;  // of a unit
};

// What a block of K costs on a tile `bn` wide, in columns: a pair's time goes
// with the operands' bytes, which the tiles' 256 rows share (4096 x 16384 x 4096:
// 14.0 us a round of 128 columns, 20.9 of 256). Few tokens leave the SMs waiting
// for the weights, and a little for each tile: 1 x 131072 x 4096 took 168 us by
// six tiles of 144 columns a CTA and 161 by four of 224, 77 x 50001 x 2001 52.5
// by three of 112 and 43.8 by two of 176.
int64_t tile_cost(int cg, int bn) { return cg == 2 ? bn + 160 : bn + 16; }

// The units of a product of A (M x K) and B (N x K), either of which may have its
// rows or K contiguous (mn).
template <int CG>
gemm_status_t shape_job(Job *job, int bn, int splits, int64_t M, int64_t N, int64_t K, int a_mn, int b_mn)
{
    constexpr int BK = kHeadBK<CG>;
    HeadJob &j = job->j;
    const int64_t tiles_m = (M + 128 * CG - 1) / (128 * CG), tiles_n = (N + bn - 1) / bn;
    const int64_t kb = (K + BK - 1) / BK, unit = (kb + splits - 1) / splits, parts = (kb + unit - 1) / unit;
    if (tiles_m * tiles_n * parts > kSizeLimit / 2)  // a cluster's last step may pass the end once
        return GEMM_ERR_UNSUPPORTED;
    j.M = static_cast<int>(M);
    j.N = static_cast<int>(N);
    j.K = static_cast<int>(K);
    j.tiles_m = static_cast<int>(tiles_m);
    j.tiles_n = static_cast<int>(tiles_n);
    j.units = static_cast<int>(tiles_m * tiles_n * parts);
    j.group_m = static_cast<int>(std::min<int64_t>(8, tiles_m));
    j.by_tiles = divisor(tiles_m * tiles_n);
    j.by_group = divisor(j.group_m * tiles_n);
    j.by_rows = divisor(j.group_m);
    j.by_last_rows = divisor(tiles_m % j.group_m ? tiles_m % j.group_m : j.group_m);
    j.kb_all = static_cast<int>(kb);
    j.kb_unit = static_cast<int>(unit);
    j.kb_part = static_cast<int>(unit);
    j.bn = bn;
    // the last tile of a row: as many boxes of 64 columns as it needs (where B's
    // K is contiguous, the stage's layout goes with the width, which stays)
    j.bn_last = b_mn ? static_cast<int>(round_up(N - (tiles_n - 1) * bn, 64 * CG)) : bn;
    j.a_mn = a_mn;
    j.b_mn = b_mn;
    // an epilogue that no other unit's products cover costs about four blocks
    job->cost = (unit + 4) * ((tiles_n - 1) * tile_cost(CG, bn) + tile_cost(CG, j.bn_last)) / tiles_n;
    return GEMM_OK;
}

// Its operands' maps.
template <int CG>
gemm_status_t map_operands(Job *job, int in_bf16, const Operand &A, const Operand &B, int a_rows)
{
    constexpr int BK = kHeadBK<CG>;
    const HeadJob &j = job->j;
    const gemm_status_t s = encode_16(&job->a, in_bf16, A.ptr, j.a_mn, j.M, j.K, A.ld, a_rows, BK);
    return s == GEMM_OK ? encode_16(&job->b, in_bf16, B.ptr, j.b_mn, j.N, j.K, B.ld, j.bn / CG, BK) : s;
}

template <int CG, int MODE>
std::atomic<uint64_t> head_attribute_set[2] = {{0}, {0}};

// Deals the units of the jobs, the longest first, out to the clusters: the jobs
// are put into that order. Returns the clusters.
int64_t deal_units(Job *jobs, int n, int64_t slots)
{
    std::sort(jobs, jobs + n, [](const Job &x, const Job &y) { return x.cost > y.cost; });
    int64_t units = 0;
    for (int i = 0; i < n; ++i)
        units += jobs[i].j.units;
    const int64_t clusters = std::min<int64_t>(units, slots);
    int64_t behind = 0, gap = 0;  // clusters from `behind` on have `gap` less to do
    for (int i = 0; i < n; ++i) {
        HeadJob &j = jobs[i].j;
        const int64_t cost = jobs[i].cost, late = clusters - behind;
        j.behind = static_cast<int>(behind);
        j.extra = behind > 0 ? static_cast<int>((gap + cost / 2) / cost) : 0;
        const int64_t rest = j.units - j.extra * late;
        if (rest <= 0) {
            gap = std::max<int64_t>(0, gap - j.units / late * cost);  // they may have been rounded up past it
        } else if (rest % clusters != 0) {
            behind = rest % clusters;
            gap = cost;
        } else {
            behind = gap = 0;
        }
    }
    return clusters;
}

int64_t cluster_slots(int cg, int sms) { return std::max(1, sms / cg); }

// Deals the units out and launches the jobs together.
template <int CG, int MODE>
gemm_status_t launch_head(HeadParams p, Job *jobs, int n, int sms, cudaStream_t st)
{
    constexpr int BK = kHeadBK<CG>;
    const int64_t clusters = deal_units(jobs, n, cluster_slots(CG, sms));
    int64_t longest = 0;
    int bn = 0;
    HeadMaps maps;
    for (int i = 0; i < n; ++i) {
        longest = std::max<int64_t>(longest, jobs[i].j.kb_unit);
        bn = std::max(bn, jobs[i].j.bn);
    }
    for (int i = 0; i < kMaxJobs; ++i) {
        const Job &job = jobs[i < n ? i : 0];
        p.jobs[i] = job.j;
        maps.a[i] = job.a;
        maps.b[i] = job.b;
        maps.d[i] = job.d;
    }
    p.num_jobs = n;
    p.b_rows = bn / CG;
    int ms = 0;
    p.inject = host_take_injection(&ms);
    // a role may wait for another to walk all of a unit's K: 10 us a block beside 2 s
    p.timeout_ns = ms > 0 ? static_cast<unsigned long long>(ms) * 1000000ull : 2000000000ull + static_cast<unsigned long long>(longest) * 10000ull;
    const int stage_bytes = (p.a_rows + p.b_rows) * BK * 2;
    const int rest = (MODE == kForward ? kHeadShares : kHeadStageBytes) + kHeadTail;
    p.stages = std::min(kHeadMaxStages, (kHeadSmem - rest) / stage_bytes);
    const int smem = p.stages * stage_bytes + rest + 1024;
    auto kern = head_kernel<CG, MODE>;
    if constexpr (MODE == kBackwardParts) {
        // an inc of more than the launch has would wait for ever
        static const bool regs_ok = [&] {
            cudaFuncAttributes at;
            return cudaFuncGetAttributes(&at, kern) == cudaSuccess && at.numRegs == kBackLaunchRegs;
        }();
        if (!regs_ok)
            return GEMM_ERR_UNSUPPORTED;
    }
    if (ensure_smem_attribute(kern, kHeadSmem + 1024, head_attribute_set<CG, MODE>) != cudaSuccess)
        return GEMM_ERR_CUDA;
    return host_launch(kern, static_cast<unsigned>(clusters * CG), kHeadThreads<CG, MODE>, static_cast<size_t>(smem), st, CG == 2 ? 2u : 0u, maps, p);
}

// Columns of the tiles of the logits: 256, or the width whose rounds of the grid
// cost least where there are few. A tile of few rows of A is at least so wide
// that the 128 rows the tensor cores read of a stage lie inside it.
int logit_columns(int cg, int64_t T, int64_t V, int a_rows, int step, int sms)
{
    const int64_t slots = cluster_slots(cg, sms), tiles_m = (T + 128 * cg - 1) / (128 * cg);
    const int least = cg == 2 ? 128 : std::max(64, 128 - a_rows);
    int best = 256;
    int64_t best_cost = 0;
    for (int bn = 256; bn >= least; bn -= step) {
        const int64_t rounds = (tiles_m * ((V + bn - 1) / bn) + slots - 1) / slots, cost = rounds * tile_cost(cg, bn);
        if (best_cost == 0 || cost < best_cost) {
            best_cost = cost;
            best = bn;
        }
    }
    return best;
}

// Vocabulary columns of a piece, parts of dX, and the places of all that in the
// workspace.
struct BackPlan {
    int cg;
    int64_t piece, pieces, ldp;  // columns of a piece (a multiple of 256 but for the only one), their number, elements of its rows
    int64_t ldk;                 // elements of a row of X's copy and of dX's parts
    int dx_bn, dx_splits;
    size_t xs, dl[2], parts, bytes;  // offsets
};

// How the vocabulary is cut into pieces of at most `columns`, and the bytes of dl.
struct Pieces {
    int64_t piece, pieces, ldp;
    size_t dl_bytes;  // one piece's
};

Pieces cut_vocabulary(int64_t T, int64_t V, int64_t columns)
{
    Pieces p;
    p.pieces = (V + columns - 1) / columns;
    p.piece = p.pieces == 1 ? V : round_up((V + p.pieces - 1) / p.pieces, 256);
    p.pieces = (V + p.piece - 1) / p.piece;
    p.ldp = round_up(p.piece, 64);
    p.dl_bytes = static_cast<size_t>(round_up(T * p.ldp * 2, 256));
    return p;
}

// Rows of a tile and elements of K in a block, and the most parts that dX is cut
// into: two for each cluster that its tiles leave without one.
struct DxTiles {
    int cg, bn, bk;
    int64_t slots, tiles, most_splits;
};

// Up to 128 tokens have tiles of single CTAs: one row of tiles, whose columns twice
// as many share as there are pairs. More have pairs, since two rows of single
// tiles would read the weights twice. By the other of the two, at V 131072, K 2048: forward 64 tokens
// 99.0 us instead of 88.4, 128 99.7 (89.0), 129 116.7 (100.3), 256 127.5 (103.6);
// backward 64 338.6 (320.2), 128 352.0 (333.1), 129 394 (367), 256 439 (389). At V
// 32768, K 1024 forward 128 18.9 (14.9), 129 20.4 (18.5), 257 25.8 (27.3), 384 27.2
// both ways, 512 33.6 (29.4).
DxTiles dx_tiles(int64_t T, int64_t K, int sms)
{
    DxTiles d;
    d.cg = T <= 128 ? 1 : 2;
    d.bn = K <= 128 ? 128 : 256;
    d.bk = d.cg == 2 ? kHeadBK<2> : kHeadBK<1>;
    d.slots = cluster_slots(d.cg, sms);
    d.tiles = (T + 128 * d.cg - 1) / (128 * d.cg) * ((K + d.bn - 1) / d.bn);
    d.most_splits = std::max<int64_t>(1, 2 * d.slots / d.tiles);
    return d;
}

// Room for the most parts of dX that any piece would have: narrower pieces, of
// which some have more, never need more room than wider ones.
size_t parts_bytes(int64_t T, int64_t V, int64_t K, int sms)
{
    const DxTiles d = dx_tiles(T, K, sms);
    return static_cast<size_t>(round_up(T * round_up(K, 8) * 4 * std::min(d.most_splits, (V + d.bk - 1) / d.bk), 256));
}

BackPlan back_plan(int64_t T, int64_t V, int64_t K, int64_t columns, int sms)
{
    BackPlan b = {};
    const Pieces cut = cut_vocabulary(T, V, columns);
    const DxTiles d = dx_tiles(T, K, sms);
    b.cg = d.cg;
    b.piece = cut.piece;
    b.pieces = cut.pieces;
    b.ldp = cut.ldp;
    b.ldk = round_up(K, 8);
    b.dx_bn = d.bn;
    // dX has few tiles with long sums over the piece: in parts, where one would
    // take more than a third of what a cluster has to do in all
    const int rows = 128 * b.cg;
    auto blocks = [&](int64_t n) { return (n + d.bk - 1) / d.bk; };
    auto tiles = [&](int64_t m, int64_t n, int bn) { return (m + rows - 1) / rows * ((n + bn - 1) / bn); };
    const int64_t kb = blocks(b.piece);
    const int64_t work = d.tiles * kb + tiles(b.piece, K, b.dx_bn) * (blocks(T) + 4) + (b.pieces > 1 ? tiles(T, b.piece, 256) * (blocks(K) + 4) : 0);
    const int64_t most = std::max<int64_t>(8, work / d.slots / 3);
    const int64_t wanted = std::min<int64_t>((kb + most - 1) / most, d.most_splits), unit = (kb + wanted - 1) / wanted;
    b.dx_splits = static_cast<int>((kb + unit - 1) / unit);
    size_t at = 256;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    b.xs = take(static_cast<size_t>(T) * b.ldk * 2);
    b.dl[0] = take(cut.dl_bytes);
    b.dl[1] = b.pieces > 1 ? take(cut.dl_bytes) : b.dl[0];
    b.parts = take(parts_bytes(T, V, K, sms));
    b.bytes = at;
    return b;
}

// Widest pieces that are taken: a piece's dl has 256 MB at most. Few tokens wait
// for memory, and have all of the vocabulary in one piece: pieces small enough
// to stay in L2 from one launch to the next left most SMs without tiles (1 x
// 131072 x 4096: 1140 us by tiles in pieces of 8192, 607 in one; 128 x 131072 x
// 2048: 499 and 338).
constexpr int64_t kDlElements = int64_t(1) << 27;

int64_t widest_piece(int64_t T) { return std::max<int64_t>(256, kDlElements / std::max<int64_t>(T, 1) / 256 * 256); }

// What both calls check of their shape.
gemm_status_t check_head(int in_type, int64_t T, int64_t V, int64_t K, const void *X, int64_t ldx, const void *W, int64_t ldw,
                         const int32_t *targets)
{
    if ((in_type != 0 && in_type != 1) || !valid_size(T) || !valid_size(V) || !valid_size(K) || V < 1 || K < 1)
        return GEMM_ERR_INVALID_ARG;
    if (T == 0)
        return GEMM_OK;
    if (!X || !W || !targets || ldx < K || ldw < K || !valid_stride(ldx, 2) || !valid_stride(ldw, 2))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(X, 16) || !aligned_to(W, 16) || ldx % 8 != 0 || ldw % 8 != 0 || !aligned_to(targets, 4))
        return GEMM_ERR_ALIGNMENT;
    if (!countable(T) || !countable(V) || !countable(K))
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// Room for partial softmaxes on any GPU: one for each tile, which has at least 64
// columns, or where tokens have CTA pairs 128 (and for the most tokens that have none).
size_t forward_bytes(int64_t T, int64_t V)
{
    const size_t narrow = static_cast<size_t>(std::min<int64_t>(T, 128)) * static_cast<size_t>((V + 63) / 64) * sizeof(float2);
    return T <= 128 ? narrow : std::max(narrow, static_cast<size_t>(T) * static_cast<size_t>((V + 127) / 128) * sizeof(float2));
}

// The forward product, and the rows of X's places in a stage.
template <int CG>
gemm_status_t forward_job(Job *job, int64_t T, int64_t V, int64_t K, int sms, int *a_rows)
{
    *a_rows = CG == 2 ? 128 : static_cast<int>(std::min<int64_t>(128, round_up(T, 8)));
    const gemm_status_t s = shape_job<CG>(job, logit_columns(CG, T, V, *a_rows, CG == 2 ? 32 : 16, sms), 1, T, V, K, 0, 0);
    job->j.epi = kEpiSoftmax;
    job->j.kb_part = static_cast<int>(sum_part(CG, T) / kHeadBK<CG>);
    return s;
}

template <int CG>
gemm_status_t run_forward(HeadParams p, int64_t T, int64_t V, int64_t K, int in_type, const Operand &X, const Operand &W, int *tiles, int sms,
                          cudaStream_t st)
{
    Job job;
    if (forward_job<CG>(&job, T, V, K, sms, &p.a_rows) != GEMM_OK)
        return GEMM_ERR_UNSUPPORTED;
    const gemm_status_t s = map_operands<CG>(&job, in_type, X, W, p.a_rows);
    if (s != GEMM_OK)
        return s;
    job.d = job.a;
    *tiles = job.j.tiles_n;
    return launch_head<CG, kForward>(p, &job, 1, sms, st);
}

constexpr int kFewTokens = 2;

bool few_tokens(int64_t T, int64_t K) { return T <= kFewTokens && K <= 8 * kFewThreads; }

size_t few_bytes(int64_t T, int64_t K) { return static_cast<size_t>(kFewBlocks) * T * round_up(K, 8) * 4; }

// Most room for dl that up to T tokens take by pieces of at most `columns` (a
// multiple of 256). Pieces of one width need more for more tokens, up to as many
// as may have that width; the next width may then need less.
size_t most_dl(int64_t T, int64_t V, int64_t columns)
{
    auto bytes = [&](int64_t t, int64_t c) {
        const Pieces p = cut_vocabulary(t, V, c);
        return p.dl_bytes * (p.pieces > 1 ? 2 : 1);
    };
    size_t most = bytes(T, std::min(columns, widest_piece(T)));
    while (true) {
        const Pieces p = cut_vocabulary(1, V, columns);
        const int64_t last = kDlElements / round_up(p.piece, 256);  // tokens that may have pieces so wide
        if (last >= T)
            return most;
        if (p.pieces > 1)  // two of them fill the limit, as all narrower ones may
            return std::max(most, static_cast<size_t>(2 * 2 * kDlElements));
        if (last > 0)
            most = std::max(most, bytes(last, columns));
        columns = widest_piece(last + 1);
    }
}

// The same of dX's parts, whose number falls where a row of tiles begins, and by
// half where tokens have tiles of CTA pairs.
size_t most_parts(int64_t T, int64_t V, int64_t K, int sms)
{
    size_t most = parts_bytes(T, V, K, sms);
    for (int64_t rows = 128; rows < T; rows += rows == 128 ? 128 : 256) {
        most = std::max(most, parts_bytes(rows, V, K, sms));
        if (rows > 128 && dx_tiles(rows, K, sms).most_splits == 1)
            break;  // from here on one part, of more and more rows
    }
    return most;
}

// What the backward call asks for, for T tokens and for fewer.
size_t back_bytes(int64_t T, int64_t V, int64_t K, int64_t columns, int sms)
{
    if (few_tokens(T, K))
        return few_bytes(T, K);
    const int64_t all = round_up(V, 256), wide = columns ? std::min(all, round_up(columns, 256)) : all;
    const size_t tiles = 256 + static_cast<size_t>(round_up(T * round_up(K, 8) * 2, 256)) + most_dl(T, V, wide) + most_parts(T, V, K, sms);
    return few_tokens(1, K) ? std::max(tiles, few_bytes(kFewTokens, K)) : tiles;
}

// The plan of a call: the widest pieces that its workspace has room for. The
// only piece has one dl, and may need less than two pieces do.
BackPlan fit_plan(int64_t T, int64_t V, int64_t K, size_t workspace_bytes, int sms)
{
    int64_t low = 1, high = std::min(round_up(V, 256), widest_piece(T)) / 256;
    if (back_plan(T, V, K, 256 * high, sms).bytes <= workspace_bytes)
        low = high;
    else
        high = std::max<int64_t>(1, high - 1);
    while (low < high) {
        const int64_t mid = (low + high + 1) / 2;
        if (back_plan(T, V, K, 256 * mid, sms).bytes <= workspace_bytes)
            low = mid;
        else
            high = mid - 1;
    }
    return back_plan(T, V, K, 256 * low, sms);
}

// The arguments of a backward call that its launches need.
struct BackArgs {
    int in_type;
    int64_t T, V, K;
    Operand X, W;
    void *dX, *dW;
    int dx_type, dw_type;
    int64_t lddx, lddw;
    bool accumulate;
    uint8_t *ws;
};

template <typename I, int TT>
std::atomic<uint64_t> few_attribute_set[2] = {{0}, {0}};

template <typename I, int TT>
gemm_status_t launch_few(FewParams p, int groups, cudaStream_t st)
{
    const size_t smem = groups > 1 ? static_cast<size_t>(TT) * 8 * p.x_threads * 4 : 0;
    if (ensure_smem_attribute(head_few_kernel<I, TT>, TT * 4 * 8 * kFewThreads, few_attribute_set<I, TT>) != cudaSuccess)
        return GEMM_ERR_CUDA;
    return host_launch(head_few_kernel<I, TT>, kFewBlocks, dim3(p.x_threads, groups), smem, st, 0, p);
}

gemm_status_t run_few(const BackArgs &g, FewParams p, cudaStream_t st)
{
    p.x = g.X.ptr;
    p.w = g.W.ptr;
    p.dw = g.dW;
    p.parts = g.dX ? reinterpret_cast<float *>(g.ws) : nullptr;
    p.ldx = g.X.ld;
    p.ldw = g.W.ld;
    p.lddw = g.lddw;
    p.ld_parts = round_up(g.K, 8);
    p.T = static_cast<int>(g.T);
    p.V = static_cast<int>(g.V);
    p.K = static_cast<int>(g.K);
    p.x_threads = static_cast<int>(round_up((g.K + 7) / 8, 32));
    p.dw_type = g.dw_type;
    p.accumulate = g.accumulate;
    // barriers 1 to 15 are the groups' own; those of one warp need none
    const int groups = kFewThreads / p.x_threads;
    gemm_status_t s;
    if (g.in_type == 1)
        s = g.T == 1 ? launch_few<__nv_bfloat16, 1>(p, groups, st) : launch_few<__nv_bfloat16, 2>(p, groups, st);
    else
        s = g.T == 1 ? launch_few<__half, 1>(p, groups, st) : launch_few<__half, 2>(p, groups, st);
    if (s != GEMM_OK || !g.dX)
        return s;
    return with_type(g.dx_type, [&](auto tag) {
        using D = decltype(tag);
        return host_launch(head_few_sum_kernel<D>, dim3(static_cast<unsigned>((g.K + 31) / 32), static_cast<unsigned>(g.T)), 256, 0, st, 0, p.parts,
                           kFewBlocks, p.ld_parts, p.T, p.K, static_cast<D *>(g.dX), g.lddx);
    });
}

// The products of one launch, in the order dX, dW, dl (those that it has): piece
// i's gradients, and the next piece's dl. Piece -1 has dl alone.
struct PieceJobs {
    Job jobs[kMaxJobs];
    int n = 0;
    Job *dx = nullptr, *dw = nullptr, *dl = nullptr;
    int a_rows;
    int64_t v0, cols, w0, next;  // the piece's first column and its columns, the next one's
};

template <int CG>
gemm_status_t piece_jobs(PieceJobs *q, const BackPlan &b, int64_t i, int64_t T, int64_t V, int64_t K, bool want_x, bool want_w, int sms)
{
    gemm_status_t s;
    q->v0 = i * b.piece;
    q->cols = std::min(b.piece, V - q->v0);
    // dl alone: places of few rows leave the stages to the weights
    q->a_rows = CG == 1 && i < 0 ? static_cast<int>(std::min<int64_t>(128, round_up(T, 8))) : 128;
    if (i >= 0 && want_x) {
        q->dx = &q->jobs[q->n++];
        if ((s = shape_job<CG>(q->dx, b.dx_bn, b.dx_splits, T, K, q->cols, 0, 1)) != GEMM_OK)
            return s;
        q->dx->j.epi = kEpiProduct;
    }
    if (i >= 0 && want_w) {
        q->dw = &q->jobs[q->n++];
        if ((s = shape_job<CG>(q->dw, b.dx_bn, 1, q->cols, K, T, 1, 1)) != GEMM_OK)
            return s;
        q->dw->j.epi = kEpiProduct;
    }
    if (i + 1 < b.pieces) {
        q->dl = &q->jobs[q->n++];
        q->w0 = (i + 1) * b.piece;
        q->next = std::min(b.piece, V - q->w0);
        // by its own rounds of the grid, where it has a launch to itself or too few wide tiles for all clusters
        const int64_t wide = (T + 128 * CG - 1) / (128 * CG) * ((q->next + 255) / 256);
        const int bn = q->n == 1 || wide < 2 * sms / CG ? logit_columns(CG, T, q->next, q->a_rows, 64, sms) : 256;
        if ((s = shape_job<CG>(q->dl, bn, 1, T, q->next, K, 0, 0)) != GEMM_OK)
            return s;
        q->dl->j.epi = kEpiLogitGrad;
        q->dl->j.kb_part = static_cast<int>(sum_part(CG, T) / kHeadBK<CG>);
        q->dl->j.v0 = static_cast<int>(q->w0);
    }
    return GEMM_OK;
}

// One launch for each piece: its gradients and the next piece's dl, which do not
// wait for one another, so that the units of one product fill what the rounds of
// the others leave of the grid.
template <int CG>
gemm_status_t run_backward(HeadParams p, const BackArgs &g, const BackPlan &b, int sms, cudaStream_t st)
{
    const int ew = type_bytes(g.dw_type);
    float *parts = reinterpret_cast<float *>(g.ws + b.parts);
    auto weights = [&](int64_t v) { return Operand{static_cast<const char *>(g.W.ptr) + v * g.W.ld * 2, g.W.ld}; };
    for (int64_t i = -1; i < b.pieces; ++i) {
        PieceJobs q;
        gemm_status_t s = piece_jobs<CG>(&q, b, i, g.T, g.V, g.K, g.dX != nullptr, g.dW != nullptr, sms);
        if (s != GEMM_OK)
            return s;
        p.a_rows = q.a_rows;
        const Operand dl = {i >= 0 ? g.ws + b.dl[i & 1] : nullptr, b.ldp};
        if (q.dx) {
            if ((s = map_operands<CG>(q.dx, g.in_type, dl, weights(q.v0), 128)) != GEMM_OK)
                return s;
            const bool last = i == b.pieces - 1 && b.dx_splits == 1;
            HeadJob &j = q.dx->j;
            j.out_type = last ? g.dx_type : GEMM_OUT_F32;
            j.scaled = last;
            j.slot_rows = g.T;
            j.c_raw = i > 0 ? parts : nullptr;
            j.ld_raw = b.ldk;
            j.c_typed = nullptr;
            j.ld_typed = 0;
            j.whole = static_cast<int>(last ? whole_words(g.K, g.dx_type) : b.ldk);
            j.d = g.dX;
            j.ldd = g.lddx;
            if ((s = encode_out(&q.dx->d, j.out_type, last ? g.dX : parts, g.T, j.whole, last ? g.lddx : b.ldk, last ? 1 : b.dx_splits)) != GEMM_OK)
                return s;
        }
        if (q.dw) {
            if ((s = map_operands<CG>(q.dw, g.in_type, dl, {g.ws + b.xs, b.ldk}, 128)) != GEMM_OK)
                return s;
            char *o = static_cast<char *>(g.dW) + q.v0 * g.lddw * ew;
            HeadJob &j = q.dw->j;
            j.out_type = g.dw_type;
            j.scaled = 1;
            j.slot_rows = 0;
            j.c_raw = nullptr;
            j.ld_raw = 0;
            j.c_typed = g.accumulate ? o : nullptr;
            j.ld_typed = g.lddw;
            j.whole = static_cast<int>(whole_words(g.K, g.dw_type));
            j.d = o;
            j.ldd = g.lddw;
            if ((s = encode_out(&q.dw->d, g.dw_type, o, q.cols, j.whole, g.lddw)) != GEMM_OK)
                return s;
        }
        if (q.dl) {
            if ((s = map_operands<CG>(q.dl, g.in_type, g.X, weights(q.w0), q.a_rows)) != GEMM_OK ||
                (s = encode_out(&q.dl->d, g.in_type == 1 ? GEMM_OUT_BF16 : GEMM_OUT_F16, g.ws + b.dl[(i + 1) & 1], g.T, round_up(q.next, 8), b.ldp)) !=
                    GEMM_OK)
                return s;
        }
        const bool by_parts = q.dl && q.dl->j.kb_part < q.dl->j.kb_all;
        s = by_parts ? launch_head<CG, kBackwardParts>(p, q.jobs, q.n, sms, st) : launch_head<CG, kBackward>(p, q.jobs, q.n, sms, st);
        if (s != GEMM_OK)
            return s;
    }
    return GEMM_OK;
}

// The units of one launch in the order in which its clusters take them: for each
// the cluster, the product (0 dX, 1 dW, 2 logits), and the first and end of its
// rows, columns and K.
template <int CG>
int64_t list_units(Job *jobs, int n, int sms, const int *product, int32_t *out, int64_t most)
{
    for (int i = 0; i < n; ++i)
        jobs[i].j.out_type = product[i];  // through the sort
    const int64_t clusters = deal_units(jobs, n, cluster_slots(CG, sms));
    HeadJob js[kMaxJobs];
    for (int i = 0; i < n; ++i)
        js[i] = jobs[i].j;
    int64_t count = 0;
    for (int64_t c = 0; c < clusters; ++c) {
        HeadUnits units(js, n, static_cast<int>(c), static_cast<int>(clusters));
        HeadUnit h;
        while (units.next(h)) {
            if (count < most) {
                const HeadJob &j = js[h.job];
                int32_t *o = out + 8 * count;
                auto range = [&](int first, int step, int end) {
                    *o++ = first;
                    *o++ = std::min(first + step, end);
                };
                *o++ = static_cast<int32_t>(c);
                *o++ = j.out_type;
                range(h.m_blk * 128 * CG, 128 * CG, j.M);
                range(h.n_blk * j.bn, h.n_blk == j.tiles_n - 1 ? j.bn_last : j.bn, j.N);
                range(h.kb0 * kHeadBK<CG>, (h.kb1 - h.kb0) * kHeadBK<CG>, j.K);
            }
            ++count;
        }
    }
    return count;
}

template <int CG>
int64_t launch_units(int64_t T, int64_t V, int64_t K, int64_t columns, int sms, int64_t piece, int want, int32_t *out, int64_t most)
{
    if (want == 0) {
        Job job;
        int a_rows, product = 2;
        return forward_job<CG>(&job, T, V, K, sms, &a_rows) == GEMM_OK ? list_units<CG>(&job, 1, sms, &product, out, most) : -1;
    }
    const int64_t widest = std::min(round_up(V, 256), widest_piece(T));
    const BackPlan b = back_plan(T, V, K, columns ? std::min(widest, round_up(columns, 256)) : widest, sms);
    PieceJobs q;
    if (piece < -1 || piece >= b.pieces || piece_jobs<CG>(&q, b, piece, T, V, K, want & 1, want & 2, sms) != GEMM_OK)
        return -1;
    int products[kMaxJobs], n = 0;
    if (q.dx)
        products[n++] = 0;
    if (q.dw)
        products[n++] = 1;
    if (q.dl)
        products[n++] = 2;
    return list_units<CG>(q.jobs, n, sms, products, out, most);
}

}  // namespace

// ---------------------------------------------------------------- C ABI

extern "C" {

size_t gemm_cross_entropy_workspace_size(int64_t T, int64_t V)
{
    return T < 1 || V < 1 || !countable(T) || !countable(V) ? 0 : forward_bytes(T, V);
}

gemm_status_t gemm_cross_entropy(int in_type, int64_t T, int64_t V, int64_t K, const void *X, int64_t ldx, const void *W, int64_t ldw,
                                 const int32_t *targets, float *losses, float *lse, void *workspace, size_t workspace_bytes,
                                 gemm_stream_t stream)
{
    gemm_status_t s = check_head(in_type, T, V, K, X, ldx, W, ldw, targets);
    if (s != GEMM_OK || T == 0)
        return s;
    if (!losses || !lse || !workspace || workspace_bytes < forward_bytes(T, V))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(losses, 4) || !aligned_to(lse, 4) || !aligned_to(workspace, 16))
        return GEMM_ERR_ALIGNMENT;
    int dev = 0, sms = 0;
    HeadParams p = {};
    if ((s = host_device(&dev, &p.status, &sms)) != GEMM_OK)
        return s;
    p.targets = targets;
    p.T = static_cast<int>(T);
    p.V = static_cast<int>(V);
    p.in_bf16 = in_type;
    p.partials = static_cast<float2 *>(workspace);
    p.picked = losses;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int parts = 0;
    s = T <= 128 ? run_forward<1>(p, T, V, K, in_type, {X, ldx}, {W, ldw}, &parts, sms, st)
                 : run_forward<2>(p, T, V, K, in_type, {X, ldx}, {W, ldw}, &parts, sms, st);
    if (s != GEMM_OK)
        return s;
    if (T <= 512)
        return host_launch(head_combine_kernel<1>, static_cast<unsigned>(T), 32 * kCombineWarps, 0, st, 0, p.partials, parts, T, targets, p.V, losses, lse);
    return host_launch(head_combine_kernel<8>, static_cast<unsigned>((T + 7) / 8), 32 * kCombineWarps, 0, st, 0, p.partials, parts, T, targets, p.V,
                       losses, lse);
}

size_t gemm_cross_entropy_backward_workspace_size(int64_t T, int64_t V, int64_t K, int64_t columns)
{
    if (T < 1 || V < 1 || K < 1 || columns < 0 || !countable(T) || !countable(V) || !countable(K))
        return 0;
    if (few_tokens(T, K))
        return few_bytes(T, K);
    int dev = 0, sms = 0;
    unsigned int *status = nullptr;
    if (host_device(&dev, &status, &sms) != GEMM_OK)
        return 0;
    return back_bytes(T, V, K, columns, sms);
}

gemm_status_t gemm_cross_entropy_backward(int in_type, int64_t T, int64_t V, int64_t K, const void *X, int64_t ldx, const void *W,
                                          int64_t ldw, const int32_t *targets, const float *lse, const float *dlosses,
                                          const float *dlse, void *dX, gemm_out_t dx_type, int64_t lddx, void *dW, gemm_out_t dw_type,
                                          int64_t lddw, int accumulate, void *workspace, size_t workspace_bytes, gemm_stream_t stream)
{
    gemm_status_t s = check_head(in_type, T, V, K, X, ldx, W, ldw, targets);
    if (s != GEMM_OK)
        return s;
    if (!valid_type(dx_type) || !valid_type(dw_type) || (!dX && !dW))
        return GEMM_ERR_INVALID_ARG;
    const int ex = type_bytes(dx_type), ew = type_bytes(dw_type);
    if ((dX && (lddx < K || !valid_stride(lddx, ex))) || (dW && (lddw < K || !valid_stride(lddw, ew))))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(dX, 16) || !aligned_to(dW, 16) || (dX && lddx * ex % 16 != 0) || (dW && lddw * ew % 16 != 0))
        return GEMM_ERR_ALIGNMENT;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (!dW || accumulate)
            return GEMM_OK;
        return host_launch(head_zero_kernel, static_cast<unsigned>(std::min<int64_t>(V, 4096)), 256, 0, st, 0, static_cast<uint8_t *>(dW),
                           lddw * ew, V, K * ew);
    }
    if (!lse || !dlosses || !workspace)
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(lse, 4) || !aligned_to(dlosses, 4) || !aligned_to(dlse, 4) || !aligned_to(workspace, 256))
        return GEMM_ERR_ALIGNMENT;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const BackArgs args = {in_type, T, V, K, {X, ldx}, {W, ldw}, dX, dW, dx_type, dw_type, lddx, lddw, accumulate != 0, ws};
    if (few_tokens(T, K)) {
        if (workspace_bytes < few_bytes(T, K))
            return GEMM_ERR_INVALID_ARG;
        FewParams f = {};
        f.targets = targets;
        f.lse = lse;
        f.dlosses = dlosses;
        f.dlse = dlse;
        return run_few(args, f, st);
    }
    int dev = 0, sms = 0;
    HeadParams p = {};
    if ((s = host_device(&dev, &p.status, &sms)) != GEMM_OK)
        return s;
    const BackPlan b = fit_plan(T, V, K, workspace_bytes, sms);
    if (b.bytes > workspace_bytes)
        return GEMM_ERR_INVALID_ARG;
    float *scale = reinterpret_cast<float *>(ws);
    const unsigned copies = dW ? static_cast<unsigned>(std::min<int64_t>((T * ((K + 7) / 8) + 2047) / 2048, 2 * sms)) : 0;
    if ((s = host_launch(head_prepare_kernel, 1 + copies, kPrepareThreads, 0, st, 0, static_cast<const uint4 *>(X), ldx / 8,
                         dW ? reinterpret_cast<uint4 *>(ws + b.xs) : nullptr, b.ldk / 8, static_cast<int>(K), T, targets,
                         static_cast<int>(V), dlosses, dlse, in_type == 1 ? 1.0f : 16384.0f, scale)) != GEMM_OK)
        return s;
    p.targets = targets;
    p.T = static_cast<int>(T);
    p.V = static_cast<int>(V);
    p.in_bf16 = in_type;
    p.lse = lse;
    p.dlosses = dlosses;
    p.dlse = dlse;
    p.scale = scale;
    s = b.cg == 1 ? run_backward<1>(p, args, b, sms, st) : run_backward<2>(p, args, b, sms, st);
    const int splits = b.dx_splits;
    if (s != GEMM_OK || !dX || splits == 1)
        return s;
    const float *parts = reinterpret_cast<const float *>(ws + b.parts);
    const int64_t items = T * ((K + 3) / 4);
    const long long stride = T * b.ldk;
    return with_type(dx_type, [&](auto tag) {
        using D = decltype(tag);
        if (splits > kSumGroups && items < int64_t(sms) * 1024)
            return host_launch(head_sum_kernel<D, kSumGroups>, static_cast<unsigned>(std::min<int64_t>((items * kSumGroups + 255) / 256, 8 * sms)), 256, 0,
                               st, 0, parts, splits, stride, b.ldk, T, static_cast<int>(K), scale, static_cast<D *>(dX), lddx);
        return host_launch(head_sum_kernel<D, 1>, static_cast<unsigned>(std::min<int64_t>((items + 255) / 256, 8 * sms)), 256, 0, st, 0, parts, splits,
                           stride, b.ldk, T, static_cast<int>(K), scale, static_cast<D *>(dX), lddx);
    });
}

gemm_status_t gemm_debug_cross_entropy_plan(int64_t T, int64_t V, int64_t K, int64_t columns, int sms, uint64_t workspace_bytes, int64_t *out)
{
    if (!out || T < 1 || V < 1 || K < 1 || columns < 0 || sms < 1 || !countable(T) || !countable(V) || !countable(K))
        return GEMM_ERR_INVALID_ARG;
    out[0] = static_cast<int64_t>(back_bytes(T, V, K, columns, sms));
    if (few_tokens(T, K)) {
        out[1] = static_cast<int64_t>(few_bytes(T, K));
        out[2] = out[3] = out[4] = out[5] = 0;
        return GEMM_OK;
    }
    const BackPlan b = fit_plan(T, V, K, static_cast<size_t>(workspace_bytes), sms);
    out[1] = static_cast<int64_t>(b.bytes);
    out[2] = b.cg;
    out[3] = b.pieces;
    out[4] = b.piece;
    out[5] = b.dx_splits;
    return GEMM_OK;
}

int64_t gemm_debug_cross_entropy_units(int64_t T, int64_t V, int64_t K, int64_t columns, int sms, int64_t piece, int want, int32_t *out,
                                       int64_t max_units)
{
    if (T < 1 || V < 1 || K < 1 || columns < 0 || sms < 1 || !countable(T) || !countable(V) || !countable(K) || want < 0 || want > 3 || max_units < 0 ||
        (max_units > 0 && !out) || (want > 0 && few_tokens(T, K)))
        return -1;
    return T <= 128 ? launch_units<1>(T, V, K, columns, sms, piece, want, out, max_units)
                    : launch_units<2>(T, V, K, columns, sms, piece, want, out, max_units);
}

}  // extern "C"
