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

#include "../../include/gemm_gb300.h"
#include "elements.cuh"
#include "gemm_kernel.cuh"
#include "host.h"
#include "launch.cuh"

using namespace g300;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kHeadWarps = 8;                      // epilogue warps: a lane quarter and half of the columns each
constexpr int kHeadThreads = 64 + 32 * kHeadWarps;
constexpr int kHeadMaxStages = 12;
constexpr int kAccStride = 256;                    // TMEM columns from one accumulator to the next
constexpr int kHeadSmem = 232448 - 1024;           // less the slack that rounds the base up to 1024 bytes

// Elements of K that the tensor cores sum for the softmax before the sum is
// added to the others in registers. Their additions truncate (every 16 elements,
// to the accumulator's 24 bits), which moves a logit towards 0 by up to half a
// part in 2^24 for each. Relative error of the losses, and time, of 8192 tokens,
// 65536 words and K = 4096 by parts of 256, 512, 1024 and all of K: 1.2e-7 (3020
// us), 2.2e-7 (2575), 4.7e-7 (2498), 2.0e-6 (2459); fp32 sums that round 5.2e-7.
constexpr int kSumPart = 512;

// What the epilogue does with the accumulator.
enum : int { kEpiSoftmax = 0, kEpiLogitGrad = 1, kEpiProduct = 2 };

// Offsets behind the stages: staging chunks, then barriers.
constexpr int kHeadStageBytes = kHeadWarps * kEpiBufBytes;
constexpr int kHeadBars = 2 * kHeadMaxStages + 4 + 2;
constexpr int kHeadTail = kHeadBars * 8 + 16;

struct HeadParams {
    int M, N, K;  // of this product: rows, columns, length of the sums
    int tiles_m, tiles_n, units;
    int kb_unit;  // K blocks of one unit: units = tiles * splits of K
    int kb_part;  // K blocks that the tensor cores sum before the epilogue takes the sum (a unit's, or fewer)
    int bn;       // columns of a tile
    int a_rows;   // rows of A that a CTA loads (all 128, or fewer for few tokens)
    int a_mn, b_mn, in_bf16;
    int stages, group_m;
    unsigned long long timeout_ns;
    int inject;
    unsigned int *status;
    // softmax and its gradient: column v0 + n of the vocabulary
    const int *targets;
    int V, v0;
    float2 *partials;  // [2 * tiles_n][M]: reference and sum, base 2
    float *picked;     // the targets' logits
    const float *lse, *dlosses, *dlse;
    float *scale;      // {what dl is multiplied by, its inverse}
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

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Elements of K in a stage.
template <int CG>
constexpr int kHeadBK = CG == 2 ? 128 : 64;

struct HeadUnit {
    int m_blk, n_blk, split, kb0, kb1;
};

// Units in rasters of group_m tile rows (as decode_tile), one split of K after another.
__device__ __forceinline__ HeadUnit head_unit(int tiles_m, int tiles_n, int group_m, int kb_unit, int kb_all, int u)
{
    HeadUnit h;
    const int tiles = tiles_m * tiles_n;
    h.split = u / tiles;
    const int local = u - h.split * tiles;
    const int per_group = group_m * tiles_n;
    const int g = local / per_group;
    const int rows = min(tiles_m - g * group_m, group_m);
    const int r = local - g * per_group;
    h.m_blk = g * group_m + r % rows;
    h.n_blk = r / rows;
    h.kb0 = h.split * kb_unit;
    h.kb1 = min(kb_all, h.kb0 + kb_unit);
    return h;
}

template <int CG>
__device__ ProducerTail head_producer(const HeadParams &p, const CUtensorMap *tmA, const CUtensorMap *tmB, uint32_t smem,
                                      uint32_t bar_full, uint32_t bar_empty, uint32_t bar_inject, uint32_t rank, const Waiter &w)
{
    constexpr int BK = kHeadBK<CG>;
    if (p.inject == kRoleProducer) {
        w.wait(bar_inject, 0u, kRoleProducer | kWaitInjected);
        return ProducerTail{0, 0, 0u};
    }
    const int tiles_m = p.tiles_m, tiles_n = p.tiles_n, units = p.units, group_m = p.group_m, kb_unit = p.kb_unit;
    const int bn = p.bn, stages = p.stages, kb_all = ceil_div_i(p.K, BK);
    const OperandBoxes box_a = operand_boxes(p.a_mn, 3, p.a_rows, BK, 2);
    const OperandBoxes box_b = operand_boxes(p.b_mn, 3, bn / CG, BK, 2);
    const uint32_t a_bytes = static_cast<uint32_t>(p.a_rows) * BK * 2, b_bytes = static_cast<uint32_t>(bn / CG) * BK * 2;
    const int nbox = max(box_a.nbox, box_b.nbox);
    const uint32_t full_target = CG == 2 ? mapa_shared(bar_full, 0) : bar_full;
    const int cluster = blockIdx.x / CG, clusters = gridDim.x / CG;
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    for (int u = cluster; u < units; u += clusters) {
        const HeadUnit h = head_unit(tiles_m, tiles_n, group_m, kb_unit, kb_all, u);
        const int m0 = (h.m_blk * CG + static_cast<int>(rank)) * 128;
        const int n0 = h.n_blk * bn + (bn / CG) * static_cast<int>(rank);
        for (int kb = h.kb0; kb < h.kb1; ++kb) {
            if (!w.wait(bar_empty + 8 * stage, phase ^ 1u, kRoleProducer | kWaitEmpty, rank != 0))
                return ProducerTail{min(issued, stages), stage, phase};
            if (rank == 0)
                mbar_arrive_expect_tx(bar_full + 8 * stage, CG * (a_bytes + b_bytes));
            const uint32_t sa = smem + static_cast<uint32_t>(stage) * (a_bytes + b_bytes);
            const uint32_t fb = full_target + 8 * stage;
            for (int b = 0; b < nbox; ++b) {
                if (b < box_a.nbox)
                    issue_box<CG>(tmA, sa, fb, box_a, b, m0, kb * BK);
                if (b < box_b.nbox)
                    issue_box<CG>(tmB, sa + a_bytes, fb, box_b, b, n0, kb * BK);
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
    const int tiles_m = p.tiles_m, tiles_n = p.tiles_n, units = p.units, group_m = p.group_m, kb_unit = p.kb_unit;
    const int bn = p.bn, stages = p.stages, kb_part = p.kb_part, kb_all = ceil_div_i(p.K, BK);
    const uint32_t idesc = make_idesc_f16(128 * CG, bn, p.in_bf16, p.a_mn, p.b_mn);
    const OperandPacking pa = operand_packing(p.a_mn, 3, p.a_rows, BK), pb = operand_packing(p.b_mn, 3, bn / CG, BK);
    const uint32_t a_bytes = static_cast<uint32_t>(p.a_rows) * BK * 2, b_bytes = static_cast<uint32_t>(bn / CG) * BK * 2;
    const uint64_t a_desc0 = make_smem_desc(smem, pa.lbo, pa.sbo, pa.swz);
    const uint64_t b_desc0 = make_smem_desc(smem + a_bytes, pb.lbo, pb.sbo, pb.swz);
    uint32_t a_off[SLICES], b_off[SLICES];
#pragma unroll
    for (int j = 0; j < SLICES; ++j) {
        a_off[j] = slice_byte_offset(p.a_mn, 3, p.a_rows, j) >> 4;
        b_off[j] = slice_byte_offset(p.b_mn, 3, bn / CG, j) >> 4;
    }
    const int cluster = blockIdx.x / CG, clusters = gridDim.x / CG;
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    for (int u = cluster; u < units; u += clusters) {
        const HeadUnit h = head_unit(tiles_m, tiles_n, group_m, kb_unit, kb_all, u);
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
                const uint64_t at = (static_cast<uint32_t>(stage) * (a_bytes + b_bytes)) >> 4;
#pragma unroll
                for (int j = 0; j < SLICES; ++j)
                    mma_f16<CG>(d, a_desc0 + at + a_off[j], b_desc0 + at + b_off[j], idesc, ((kb - part) | j) != 0);
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

// This thread's 32 values of a row from TMEM.
__device__ __forceinline__ void load_acc32(uint32_t taddr, float (&v)[32])
{
    uint32_t r[32];
    tmem_ld_32x32b_x32(taddr, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = __uint_as_float(r[i]);
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

    __device__ __forceinline__ void add(const float (&v)[32])
    {
        float m = v[0];
#pragma unroll
        for (int i = 1; i < 32; ++i)
            m = fmaxf(m, v[i]);
        const float top = fmaxf(r, m * kLog2e);
        const float ref = fabsf(top) == INFINITY ? 0.0f : top;
        float t[4] = {};
#pragma unroll
        for (int i = 0; i < 32; ++i)
            t[i & 3] += ex2(fmaf(v[i], kLog2e, -ref));
        s = s * ex2(r - ref) + ((t[0] + t[1]) + (t[2] + t[3]));
        r = top == INFINITY ? 0.0f : top;
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

__device__ __forceinline__ RowGrad row_grad(const HeadParams &p, int row)
{
    RowGrad g;
    if (row < p.M) {
        const int y = __ldcg(p.targets + row);
        g.live = static_cast<unsigned>(y) < static_cast<unsigned>(p.V);
        if (g.live) {
            const float by = __ldcg(p.scale), d = __ldcg(p.dlosses + row), z = p.dlse ? __ldcg(p.dlse + row) : 0.0f;
            g.a = (d + z) * by;
            g.b = d * by;
            g.lse2 = __ldcg(p.lse + row) * kLog2e;
            g.target = y - p.v0;
        }
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
// chunk (SW128 rows) and on to global memory by TMA. A TMA store writes whole
// 16-byte words, also the one in which a row ends, so that the map ends before
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

// A chunk in the output's type.
template <int CW>
__device__ __forceinline__ void pack_chunk(const float (&v)[CW], int out_type, uint32_t (&o)[32])
{
    if constexpr (CW == 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            o[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            uint32_t four[4];
            pack_out(v + 8 * u, out_type, four);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[4 * u + i] = four[i];
        }
    }
}

template <int CG, int EPI, int CW>
__device__ void head_epilogue(const HeadParams &p, const CUtensorMap *tmD, uint32_t sbuf, uint32_t bar_acc_full,
                              uint32_t bar_acc_empty, uint32_t tmem, uint32_t rank, int warp, int lane, const Waiter &w)
{
    constexpr int BK = kHeadBK<CG>;
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int tiles_m = p.tiles_m, tiles_n = p.tiles_n, units = p.units, group_m = p.group_m, kb_unit = p.kb_unit;
    const int M = p.M, N = p.N, bn = p.bn, kb_all = ceil_div_i(p.K, BK);
    const uint32_t acc_empty_target = CG == 2 ? mapa_shared(bar_acc_empty, 0) : bar_acc_empty;
    const int cluster = blockIdx.x / CG, clusters = gridDim.x / CG;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = cluster; u < units; u += clusters) {
        const HeadUnit h = head_unit(tiles_m, tiles_n, group_m, kb_unit, kb_all, u);
        const int m0 = (h.m_blk * CG + static_cast<int>(rank)) * 128 + 32 * q;
        const int row = m0 + lane;
        const int n0 = h.n_blk * bn, cols = min(bn, N - n0);
        RowGrad g;
        int y = -1;
        if constexpr (EPI == kEpiLogitGrad)
            g = row_grad(p, row);
        if constexpr (EPI == kEpiSoftmax)
            y = row < M ? __ldcg(p.targets + row) - n0 : -1;
        // waits for an accumulator, and hands it back
        auto take = [&]() {
            const bool ok = w.wait(bar_acc_full + 8 * acc, acc_phase, kRoleEpilogue | kWaitAccFull, rank != 0);
            tc_fence_after_sync();
            return __all_sync(0xffffffffu, ok) != 0;
        };
        auto release = [&]() {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2)
                    mbar_arrive_cluster(acc_empty_target + 8 * acc);
                else
                    mbar_arrive(bar_acc_empty + 8 * acc);
            }
            acc ^= 1;
            acc_phase ^= acc == 0 ? 1u : 0u;
        };
        auto columns = [&](int c) {
            return tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(acc * kAccStride + c);
        };
        const bool rows = m0 < M;  // the same for the whole warp
        if constexpr (EPI == kEpiSoftmax) {
            // the parts of the sums over K, added up in registers with fp32 rounding
            float v[4][32] = {};
            for (int part = h.kb0; part < h.kb1; part += p.kb_part) {
                if (!take())
                    return;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (rows && 32 * half + 64 * j < cols) {
                        add_acc16(columns(32 * half + 64 * j), v[j]);
                        add_acc16(columns(32 * half + 64 * j + 16), v[j] + 16);
                    }
                }
                release();
            }
            RunningSoftmax sm;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 32 * half + 64 * j;
                if (rows && c < cols) {
                    if (c + 32 > cols) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[j][i] = c + i < cols ? v[j][i] : -INFINITY;
                    }
                    sm.add(v[j]);
                    const bool mine = y >= c && y < min(c + 32, cols);
                    if (__any_sync(0xffffffffu, mine)) {
                        const float x = pick32(v[j], y - c);
                        if (mine)
                            p.picked[row] = x;
                    }
                }
            }
            if (row < M)
                p.partials[static_cast<long long>(2 * h.n_blk + half) * M + row] = make_float2(sm.r, sm.s);
        } else {
            if (!take())
                return;
            if (rows) {
                for (int c = CW * half; c < cols; c += 2 * CW) {
                    float v[CW];
                    const int col = n0 + c;
                    if constexpr (EPI == kEpiLogitGrad) {
#pragma unroll
                        for (int j = 0; j < CW / 32; ++j) {
                            float x[32];
                            load_acc32(columns(c + 32 * j), x);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[32 * j + i] = g.live ? ex2(fmaf(x[i], kLog2e, -g.lse2)) * g.a : 0.0f;
                        }
                        const bool mine = g.target >= col && g.target < col + CW;
                        if (__any_sync(0xffffffffu, mine)) {
#pragma unroll
                            for (int i = 0; i < CW; ++i)
                                v[i] -= mine && g.target == col + i ? g.b : 0.0f;
                        }
                        uint32_t o[32];
                        pack_chunk<CW>(v, p.in_bf16 ? 1 : 2, o);
                        stage_and_store<CW>(o, sbuf, lane, tmD, col, m0, 0);
                    } else {
                        const float by = p.scaled ? __ldcg(p.scale + 1) : 1.0f;
#pragma unroll
                        for (int j = 0; j < CW / 32; ++j) {
                            float x[32];
                            uint32_t raw[32];
                            if (p.c_raw)
                                load_row<float, 32>(p.c_raw + (h.split * p.slot_rows + row) * p.ld_raw, col + 32 * j, N, row < M, raw);
                            __syncwarp();
                            load_acc32(columns(c + 32 * j), x);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[32 * j + i] = (p.c_raw ? x[i] + __uint_as_float(raw[i]) : x[i]) * by;
                        }
                        if (p.c_typed) {
                            uint32_t old[32];
                            if constexpr (CW == 32) {
                                load_row<float, 32>(static_cast<const float *>(p.c_typed) + row * p.ld_typed, col, N, row < M, old);
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    v[i] += __uint_as_float(old[i]);
                            } else {
                                load_row<__half, 64>(static_cast<const __half *>(p.c_typed) + row * p.ld_typed, col, N, row < M, old);
#pragma unroll
                                for (int k = 0; k < 8; ++k) {
                                    const uint32_t four[4] = {old[4 * k], old[4 * k + 1], old[4 * k + 2], old[4 * k + 3]};
                                    float f[8];
                                    unpack_in(four, p.out_type, f);
#pragma unroll
                                    for (int i = 0; i < 8; ++i)
                                        v[8 * k + i] += f[i];
                                }
                            }
                        }
                        uint32_t o[32];
                        pack_chunk<CW>(v, p.out_type, o);
                        if (col < p.whole)
                            stage_and_store<CW>(o, sbuf, lane, tmD, col, m0, h.split);
                        if (col + CW > p.whole && p.whole < N && row < M)
                            store_tail<CW>(o, static_cast<char *>(p.d) + row * p.ldd * (CW == 32 ? 4 : 2), col, p.whole, N);
                    }
                }
            }
            release();
        }
    }
    if constexpr (EPI != kEpiSoftmax) {
        if (lane == 0)
            bulk_wait_group<0>();
    }
}

// ---------------------------------------------------------------- kernel

template <int CG, int EPI>
__global__ void __launch_bounds__(kHeadThreads, 1)
    head_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmD, const __grid_constant__ HeadParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    const uint32_t rank = CG == 2 ? cluster_ctarank() & 1u : 0u;
    const int stages = p.stages;
    const uint32_t stage_bytes = static_cast<uint32_t>(p.a_rows + p.bn / CG) * kHeadBK<CG> * 2;
    const uint32_t staging = base + static_cast<uint32_t>(stages) * stage_bytes;
    const uint32_t bars = staging + (EPI == kEpiSoftmax ? 0 : kHeadStageBytes);
    const uint32_t bar_full = bars, bar_empty = bar_full + 8 * kHeadMaxStages;
    const uint32_t bar_acc_full = bar_empty + 8 * kHeadMaxStages, bar_acc_empty = bar_acc_full + 16;
    const uint32_t bar_drain = bar_acc_empty + 16, bar_inject = bar_drain + 8;
    const uint32_t misc = bar_inject + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + (misc - base));
    volatile uint32_t *abort_flag = tmem_slot + 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_acc_full + 8 * b, 1);
            mbar_init(bar_acc_empty + 8 * b, kHeadWarps * CG);
        }
        mbar_init(bar_drain, 1);
        mbar_init(bar_inject, 1);
        *abort_flag = 0u;
        fence_mbar_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        if constexpr (EPI != kEpiSoftmax)
            prefetch_tensormap(&tmD);
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
    if (warp == 0) {
        if (lane == 0) {
            // what kernels before this one wrote by ordinary stores is read by TMA
            asm volatile("fence.proxy.async;" ::: "memory");
            tail = head_producer<CG>(p, &tmA, &tmB, base, bar_full, bar_empty, bar_inject, rank, w);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            head_mma<CG>(p, base, bar_full, bar_empty, bar_acc_full, bar_acc_empty, bar_inject, tmem, w);
            mma_commit<CG>(bar_drain);
            w.drain(bar_drain, 0u, 100000000ull);
        }
    } else {
        const uint32_t sbuf = staging + static_cast<uint32_t>((warp - 2) * kEpiBufBytes);
        if constexpr (EPI == kEpiProduct) {
            if (p.out_type == 0)
                head_epilogue<CG, EPI, 32>(p, &tmD, sbuf, bar_acc_full, bar_acc_empty, tmem, rank, warp, lane, w);
            else
                head_epilogue<CG, EPI, 64>(p, &tmD, sbuf, bar_acc_full, bar_acc_empty, tmem, rank, warp, lane, w);
        } else {
            head_epilogue<CG, EPI, 64>(p, &tmD, sbuf, bar_acc_full, bar_acc_empty, tmem, rank, warp, lane, w);
        }
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

// The normaliser and loss of each token from its partial softmaxes. ROWS 32: a
// block has 32 tokens, its warps every eighth partial; ROWS 1: a block has one
// token, its threads the partials. r is a maximum over the partials, so that
// the sum is in range; the loss is taken in base 2, where the target's logit
// cancels against r before anything is rounded.
template <int ROWS>
__global__ void __launch_bounds__(256)
    head_combine_kernel(const float2 *partials, int parts, long long T, const int *targets, int V, float *losses, float *lse)
{
    __shared__ float2 part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = ROWS == 32 ? blockIdx.x * 32ll + lane : static_cast<long long>(blockIdx.x);
    const int first = ROWS == 32 ? warp : static_cast<int>(threadIdx.x), step = ROWS == 32 ? 8 : 256;
    grid_start();
    float r = -INFINITY, s = 0.0f;
    auto join = [&](float2 o) {
        const float top = fmaxf(r, o.x);
        const float ref = top == -INFINITY ? 0.0f : top;
        // a sum of 0 or infinity stays what it is whatever its reference
        const float a = r == ref || s == 0.0f || s == INFINITY ? s : s * ex2(r - ref);
        const float b = o.x == ref || o.y == 0.0f || o.y == INFINITY ? o.y : o.y * ex2(o.x - ref);
        r = top;
        s = a + b;
    };
    if (row < T) {
#pragma unroll 8
        for (int i = first; i < parts; i += step)
            join(__ldcg(partials + i * T + row));
    }
    if constexpr (ROWS == 1) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            float2 other;
            other.x = __shfl_xor_sync(0xffffffffu, r, o);
            other.y = __shfl_xor_sync(0xffffffffu, s, o);
            join(other);
        }
    }
    part[warp][lane] = make_float2(r, s);
    __syncthreads();
    if (warp != 0 || (ROWS == 1 && lane != 0) || row >= T)
        return;
    for (int i = 1; i < 8; ++i)
        join(part[i][lane]);
    const int y = __ldcg(targets + row);
    const bool live = static_cast<unsigned>(y) < static_cast<unsigned>(V);
    const float ref = r == -INFINITY ? 0.0f : r;
    const float log2s = log2f(s);
    lse[row] = live ? (ref + log2s) * kLn2 : 0.0f;
    losses[row] = live ? (fmaf(-__ldcg(losses + row), kLog2e, ref) + log2s) * kLn2 : 0.0f;
}

// What the gradients need of all tokens: block 0 finds the largest |dloss| +
// |dlse| of the live ones and sets scale = {c / largest, largest / c}, so that
// dl is at most c in magnitude whatever the caller's scaling (c = 1 for bf16,
// 2^14 for fp16, whose small probabilities would otherwise be subnormal);
// the other blocks copy X with the rows of tokens without a loss zeroed, so
// that what such a row holds (a NaN, say) does not reach dW as 0 * NaN.
__global__ void __launch_bounds__(256)
    head_prepare_kernel(const uint4 *x, long long ldx16, uint4 *xs, long long ld16, int K, long long T, const int *targets, int V,
                        const float *dlosses, const float *dlse, float c, float *scale)
{
    grid_start();
    if (blockIdx.x == 0) {
        __shared__ float top[8];
        float m = 0.0f;
        for (long long t = threadIdx.x; t < T; t += 256)
            if (static_cast<unsigned>(__ldcg(targets + t)) < static_cast<unsigned>(V))
                m = fmaxf(m, fabsf(__ldcg(dlosses + t)) + (dlse ? fabsf(__ldcg(dlse + t)) : 0.0f));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((threadIdx.x & 31) == 0)
            top[threadIdx.x >> 5] = m;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < 8; ++i)
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
    const long long all = T * words, step = (gridDim.x - 1ll) * 256;
    for (long long i = (blockIdx.x - 1ll) * 256 + threadIdx.x; i < all; i += step) {
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

// dX from the sums over parts of the vocabulary, in the order of the parts.
template <typename D>
__global__ void __launch_bounds__(256)
    head_sum_kernel(const float *parts, int n, long long stride, long long ld, long long T, int K, const float *scale, D *d, long long ldd)
{
    grid_start();
    const float by = __ldcg(scale + 1);
    const int words = (K + 3) / 4;
    const long long all = T * words, step = gridDim.x * 256ll;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < all; i += step) {
        const long long t = i / words;
        const int k = 4 * static_cast<int>(i - t * words);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j < n; ++j) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(parts + j * stride + t * ld + k));
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        D *o = d + t * ldd + k;
        const float v[4] = {s.x * by, s.y * by, s.z * by, s.w * by};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (k + j < K)
                o[j] = from_float<D>(v[j]);
    }
}

// Zeros for dW when there is no token.
__global__ void __launch_bounds__(256) head_zero_kernel(uint8_t *d, long long ld_bytes, long long rows, int row_bytes)
{
    grid_start();
    for (long long r = blockIdx.x; r < rows; r += gridDim.x)
        for (int i = 2 * static_cast<int>(threadIdx.x); i < row_bytes; i += 512)
            *reinterpret_cast<uint16_t *>(d + r * ld_bytes + i) = 0;
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
    int mn_major;
    int64_t ld;
};

// Tiles of a product: single CTAs of up to 128 rows, or pairs of 256; `bn`
// columns; K in `splits` parts.
struct HeadTiles {
    int cg, bn, splits;
};

template <int CG, int EPI>
std::atomic<uint64_t> head_attribute_set[2] = {{0}, {0}};

template <int CG, int EPI>
gemm_status_t launch_head(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &d, HeadParams &p, int sms, cudaStream_t st)
{
    constexpr int BK = kHeadBK<CG>;
    const int stage_bytes = (p.a_rows + p.bn / CG) * BK * 2;
    const int rest = (EPI == kEpiSoftmax ? 0 : kHeadStageBytes) + kHeadTail;
    p.stages = std::min(kHeadMaxStages, (kHeadSmem - rest) / stage_bytes);
    const int smem = p.stages * stage_bytes + rest + 1024;
    auto kern = head_kernel<CG, EPI>;
    if (ensure_smem_attribute(kern, kHeadSmem + 1024, head_attribute_set<CG, EPI>) != cudaSuccess)
        return GEMM_ERR_CUDA;
    const unsigned grid = static_cast<unsigned>(std::min(p.units, std::max(1, sms / CG)) * CG);
    return host_launch(kern, grid, kHeadThreads, static_cast<size_t>(smem), st, CG == 2 ? 2u : 0u, a, b, d, p);
}

// Fills in the shape of a product and launches it.
template <int EPI>
gemm_status_t run_head(HeadParams p, const HeadTiles &t, int64_t M, int64_t N, int64_t K, int in_bf16, const Operand &A, const Operand &B,
                       const CUtensorMap *d, int sms, cudaStream_t st)
{
    const int bk = t.cg == 2 ? kHeadBK<2> : kHeadBK<1>;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.bn = t.bn;
    p.a_rows = t.cg == 2 || A.mn_major ? 128 : static_cast<int>(std::min<int64_t>(128, round_up(M, 8)));
    p.a_mn = A.mn_major;
    p.b_mn = B.mn_major;
    p.in_bf16 = in_bf16;
    p.group_m = 8;
    const int64_t tiles_m = (M + 128 * t.cg - 1) / (128 * t.cg), tiles_n = (N + t.bn - 1) / t.bn;
    const int64_t kb = (K + bk - 1) / bk, unit = (kb + t.splits - 1) / t.splits, splits = (kb + unit - 1) / unit;
    if (tiles_m * tiles_n * splits > kSizeLimit)
        return GEMM_ERR_UNSUPPORTED;
    p.tiles_m = static_cast<int>(tiles_m);
    p.tiles_n = static_cast<int>(tiles_n);
    p.kb_unit = static_cast<int>(unit);
    p.kb_part = EPI == kEpiSoftmax ? kSumPart / bk : static_cast<int>(unit);
    p.units = static_cast<int>(tiles_m * tiles_n * splits);
    int ms = 0;
    p.inject = host_take_injection(&ms);
    // a role may wait for another to walk all of a unit's K: 10 us a block beside 2 s
    p.timeout_ns = ms > 0 ? static_cast<unsigned long long>(ms) * 1000000ull : 2000000000ull + static_cast<unsigned long long>(unit) * 10000ull;
    CUtensorMap a, b;
    gemm_status_t s = encode_16(&a, in_bf16, A.ptr, A.mn_major, M, K, A.ld, p.a_rows, bk);
    if (s != GEMM_OK || (s = encode_16(&b, in_bf16, B.ptr, B.mn_major, N, K, B.ld, t.bn / t.cg, bk)) != GEMM_OK)
        return s;
    const CUtensorMap &out = d ? *d : a;
    return t.cg == 2 ? launch_head<2, EPI>(a, b, out, p, sms, st) : launch_head<1, EPI>(a, b, out, p, sms, st);
}

// Rounds of the grid that `units` take, as a share of it that they fill.
double filled(int64_t units, int64_t slots) { return static_cast<double>(units) / static_cast<double>((units + slots - 1) / slots * slots); }

// Tiles of the logits: 256 columns, or the width (a multiple of `step`) whose
// rounds of the grid cost least where there are few.
HeadTiles logit_tiles(int64_t T, int64_t V, int step, int sms)
{
    HeadTiles t = {T <= 128 ? 1 : 2, 256, 1};
    const int64_t slots = std::max(1, sms / t.cg), tiles_m = (T + 128 * t.cg - 1) / (128 * t.cg);
    int64_t best = 0;
    for (int bn = 256; bn >= 128; bn -= step) {
        const int64_t units = tiles_m * ((V + bn - 1) / bn), cost = (units + slots - 1) / slots * bn;
        if (best == 0 || cost < best) {
            best = cost;
            t.bn = bn;
        }
    }
    return t;
}

// Vocabulary columns of a piece, slots for parts of dX, and the places of all
// that in the workspace.
struct BackPlan {
    int64_t piece, ldp;  // columns of a piece (a multiple of 256 but for the only one), elements of its rows
    int64_t ldk;         // elements of a row of X's copy and of dX's parts
    HeadTiles dx;
    size_t xs, dl, parts, bytes;  // offsets
};

constexpr int64_t kPieceColumns = 16384;

BackPlan back_plan(int64_t T, int64_t V, int64_t K, int64_t piece, int sms)
{
    BackPlan b = {};
    b.piece = std::min(V, piece);
    b.ldp = round_up(b.piece, 64);
    b.ldk = round_up(K, 8);
    b.dx.cg = T <= 128 ? 1 : 2;
    b.dx.bn = K <= 128 ? 128 : 256;
    const int64_t slots = std::max(1, sms / b.dx.cg);
    const int64_t tiles = (T + 128 * b.dx.cg - 1) / (128 * b.dx.cg) * ((K + b.dx.bn - 1) / b.dx.bn);
    // parts of the vocabulary that fill the grid best: each costs T K sums in
    // fp32, written and read once more
    int best = 1;
    for (int s = 2; s <= 152 && s * 512 <= b.piece; ++s)
        if (s <= 4 || tiles * s <= slots)
            if (filled(tiles * s, slots) > filled(tiles * best, slots) + 0.04)
                best = s;
    // as many as whole blocks of K make, so that no later, shorter piece has more
    const int64_t bk = b.dx.cg == 2 ? kHeadBK<2> : kHeadBK<1>, kb = (b.piece + bk - 1) / bk, unit = (kb + best - 1) / best;
    b.dx.splits = static_cast<int>((kb + unit - 1) / unit);
    size_t at = 256;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    b.xs = take(static_cast<size_t>(T) * b.ldk * 2);
    b.dl = take(static_cast<size_t>(T) * b.ldp * 2);
    b.parts = take(static_cast<size_t>(T) * b.ldk * 4 * b.dx.splits);
    b.bytes = at;
    return b;
}

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

// Room for partial softmaxes on any GPU: two for each tile of at least 128 columns.
size_t forward_bytes(int64_t T, int64_t V) { return static_cast<size_t>(T) * static_cast<size_t>((V + 127) / 128) * 2 * sizeof(float2); }

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
    const HeadTiles t = logit_tiles(T, V, 32, sms);
    p.targets = targets;
    p.V = static_cast<int>(V);
    p.partials = static_cast<float2 *>(workspace);
    p.picked = losses;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = run_head<kEpiSoftmax>(p, t, T, V, K, in_type, {X, 0, ldx}, {W, 0, ldw}, nullptr, sms, st)) != GEMM_OK)
        return s;
    const int parts = 2 * static_cast<int>((V + t.bn - 1) / t.bn);
    if (T <= 64)
        return host_launch(head_combine_kernel<1>, static_cast<unsigned>(T), 256, 0, st, 0, p.partials, parts, T, targets, p.V, losses, lse);
    return host_launch(head_combine_kernel<32>, static_cast<unsigned>((T + 31) / 32), 256, 0, st, 0, p.partials, parts, T, targets, p.V,
                       losses, lse);
}

size_t gemm_cross_entropy_backward_workspace_size(int64_t T, int64_t V, int64_t K, int64_t columns)
{
    if (T < 1 || V < 1 || K < 1 || columns < 0 || !countable(T) || !countable(V) || !countable(K))
        return 0;
    int dev = 0, sms = 0;
    unsigned int *status = nullptr;
    if (host_device(&dev, &status, &sms) != GEMM_OK)
        return 0;
    return back_plan(T, V, K, columns ? round_up(columns, 256) : kPieceColumns, sms).bytes;
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
                           lddw * ew, V, static_cast<int>(K * ew));
    }
    if (!lse || !dlosses || !workspace)
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(lse, 4) || !aligned_to(dlosses, 4) || !aligned_to(dlse, 4) || !aligned_to(workspace, 256))
        return GEMM_ERR_ALIGNMENT;
    int dev = 0, sms = 0;
    HeadParams p = {};
    if ((s = host_device(&dev, &p.status, &sms)) != GEMM_OK)
        return s;
    // the largest pieces that the workspace has room for, up to the usual ones
    BackPlan b = {};
    for (int64_t piece = kPieceColumns; piece >= 256; piece -= 256) {
        b = back_plan(T, V, K, piece, sms);
        if (b.bytes <= workspace_bytes)
            break;
    }
    if (b.bytes > workspace_bytes)
        return GEMM_ERR_INVALID_ARG;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    float *scale = reinterpret_cast<float *>(ws);
    void *xs = ws + b.xs, *dl = ws + b.dl;
    float *parts = reinterpret_cast<float *>(ws + b.parts);
    const unsigned copies = dW ? static_cast<unsigned>(std::min<int64_t>((T * ((K + 7) / 8) + 1023) / 1024, 4 * sms)) : 0;
    if ((s = host_launch(head_prepare_kernel, 1 + copies, 256, 0, st, 0, static_cast<const uint4 *>(X), ldx / 8,
                         dW ? static_cast<uint4 *>(xs) : nullptr, b.ldk / 8, static_cast<int>(K), T, targets, static_cast<int>(V), dlosses, dlse,
                         in_type == 1 ? 1.0f : 16384.0f, scale)) != GEMM_OK)
        return s;
    p.targets = targets;
    p.V = static_cast<int>(V);
    p.lse = lse;
    p.dlosses = dlosses;
    p.dlse = dlse;
    p.scale = scale;
    const int64_t pieces = (V + b.piece - 1) / b.piece;
    const int splits = b.dx.splits;
    for (int64_t i = 0; i < pieces; ++i) {
        const int64_t v0 = i * b.piece, n = std::min(b.piece, V - v0);
        const char *w = static_cast<const char *>(W) + v0 * ldw * 2;
        CUtensorMap d;
        HeadParams q = p;
        q.v0 = static_cast<int>(v0);
        if ((s = encode_out(&d, in_type == 1 ? GEMM_OUT_BF16 : GEMM_OUT_F16, dl, T, round_up(n, 8), b.ldp)) != GEMM_OK)
            return s;
        if ((s = run_head<kEpiLogitGrad>(q, logit_tiles(T, n, 64, sms), T, n, K, in_type, {X, 0, ldx}, {w, 0, ldw}, &d, sms, st)) != GEMM_OK)
            return s;
        if (dX) {
            q = p;
            const bool last = i == pieces - 1 && splits == 1;
            q.out_type = last ? dx_type : GEMM_OUT_F32;
            q.scaled = last;
            q.slot_rows = T;
            if (i > 0) {
                q.c_raw = parts;
                q.ld_raw = b.ldk;
            }
            q.whole = static_cast<int>(last ? whole_words(K, dx_type) : b.ldk);
            q.d = dX;
            q.ldd = lddx;
            if ((s = encode_out(&d, q.out_type, last ? dX : parts, T, q.whole, last ? lddx : b.ldk, last ? 1 : splits)) != GEMM_OK)
                return s;
            if ((s = run_head<kEpiProduct>(q, b.dx, T, K, n, in_type, {dl, 0, b.ldp}, {w, 1, ldw}, &d, sms, st)) != GEMM_OK)
                return s;
        }
        if (dW) {
            q = p;
            q.out_type = dw_type;
            q.scaled = 1;
            char *o = static_cast<char *>(dW) + v0 * lddw * ew;
            if (accumulate) {
                q.c_typed = o;
                q.ld_typed = lddw;
            }
            q.whole = static_cast<int>(whole_words(K, dw_type));
            q.d = o;
            q.ldd = lddw;
            if ((s = encode_out(&d, dw_type, o, n, q.whole, lddw)) != GEMM_OK)
                return s;
            const HeadTiles t = {2, K <= 128 ? 128 : 256, 1};
            if ((s = run_head<kEpiProduct>(q, t, n, K, T, in_type, {dl, 1, b.ldp}, {xs, 1, b.ldk}, &d, sms, st)) != GEMM_OK)
                return s;
        }
    }
    if (!dX || splits == 1)
        return GEMM_OK;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((T * ((K + 3) / 4) + 255) / 256, 8 * sms));
    const int k = static_cast<int>(K);
    const long long stride = T * b.ldk;
    if (dx_type == GEMM_OUT_F32)
        return host_launch(head_sum_kernel<float>, grid, 256, 0, st, 0, parts, splits, stride, b.ldk, T, k, scale, static_cast<float *>(dX), lddx);
    if (dx_type == GEMM_OUT_BF16)
        return host_launch(head_sum_kernel<__nv_bfloat16>, grid, 256, 0, st, 0, parts, splits, stride, b.ldk, T, k, scale,
                           static_cast<__nv_bfloat16 *>(dX), lddx);
    return host_launch(head_sum_kernel<__half>, grid, 256, 0, st, 0, parts, splits, stride, b.ldk, T, k, scale, static_cast<__half *>(dX), lddx);
}

}  // extern "C"
