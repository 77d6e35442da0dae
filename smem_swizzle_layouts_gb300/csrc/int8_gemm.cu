// 8-bit integer products with a scale for each row of A and each row of B:
//
//   D[m,n] = sa[m] * sb[n] * sum_k A[m,k] * B[n,k]
//
// for one matrix, or for the experts' matrices over rows of A sorted by
// expert (offsets read from device memory). Contracts are in
// include/gemm_gb300.h.
//
// sm_103a's tcgen05 has no integer kind, so the integers are widened on chip:
// TMA brings int8 tiles to shared memory, converter warps turn them into fp16
// (exact: |q| <= 128 has 8 significant bits of fp16's 11) and kind::f16 MMAs
// multiply and sum them in fp32 (exact below 2^24). The rows of B (channels)
// are the MMA's M and the rows of A (tokens) its N, so that a tile of few
// tokens still uses whole 128-row MMAs and reads every weight once.
//
// Warp roles of a CTA:
//   warp 0      TMA producer: raw int8 stages of 128 elements of K;
//   warp 1      TMEM allocator and MMA issuer;
//   warps 2-5   epilogue: accumulator (lane = channel, column = token) to D;
//   warps 6-13  converters: raw stages to fp16 stages of 64 elements of K.
// Every wait is bounded, as in gemm_kernel.cuh.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/gemm_gb300.h"
#include "gemm_kernel.cuh"
#include "host.h"
#include "launch.cuh"

namespace g300 {

constexpr int kI8Channels = 128;  // rows of B per tile (MMA M)
constexpr int kI8RawK = 128;      // elements of K per raw stage: one 128-byte swizzled row
constexpr int kI8ConvK = 64;      // elements of K per fp16 stage: one 128-byte swizzled row
constexpr int kI8ConvWarps = 8;
constexpr int kI8FirstConvWarp = 6;
constexpr int kI8Threads = 32 * (kI8FirstConvWarp + kI8ConvWarps);

enum : uint32_t {
    kRoleConvert = 6,
    kWaitRawFull = 11 << 8,
    kWaitConvEmpty = 12 << 8,
};

struct I8Params {
    int M, N, K;
    int experts;         // 0: one matrix
    const int *offsets;  // experts + 1, or null
    int tiles_n;
    const float *sa, *sb;
    void *d;
    long long ldd;
    int out_type;
    int inject;  // test hook: the role that waits on a barrier nothing arrives at
    unsigned long long timeout_ns;
    unsigned int *status;
};

// BT: tokens per tile (MMA N).
template <int BT>
struct I8Cfg {
    static constexpr int RAW_STAGES = BT >= 256 ? 2 : BT >= 128 ? 3 : 5;
    static constexpr int CONV_STAGES = 2;
    static constexpr int RAW_W = kI8Channels * kI8RawK;
    static constexpr int RAW_BYTES = RAW_W + BT * kI8RawK;
    static constexpr int CONV_W = kI8Channels * kI8ConvK * 2;
    static constexpr int CONV_BYTES = CONV_W + BT * kI8ConvK * 2;
    static constexpr int CONV_OFF = RAW_STAGES * RAW_BYTES;
    static constexpr int BAR_OFF = CONV_OFF + CONV_STAGES * CONV_BYTES;
    static constexpr int NUM_BARS = 2 * RAW_STAGES + 2 * CONV_STAGES + 4 + 2;
    static constexpr int MISC_OFF = BAR_OFF + 8 * NUM_BARS;
    static constexpr int SMEM_BASE = MISC_OFF + 16 + 1024;  // 1024: room to align the base
    static constexpr int ACC_STRIDE = BT < 32 ? 32 : BT;    // whole 32-column epilogue reads
    static constexpr int TMEM_COLS = 2 * ACC_STRIDE;
    static_assert(RAW_BYTES % 1024 == 0 && CONV_BYTES % 1024 == 0, "swizzle atoms start on 1024-byte boundaries");
    static_assert(BT % 16 == 0 && BT <= 256, "MMA N with M = 128: a multiple of 16");
    static_assert(SMEM_BASE + 2 * 4 * (GEMM_ROUTE_MAX_EXPERTS + 1) <= 232448, "shared memory per CTA");
};

// ---------------------------------------------------------------- tiles

// Tiles of `n` rows; unsigned, so that n + size may pass 2^31.
__host__ __device__ __forceinline__ int i8_tiles(int n, int size)
{
    return static_cast<int>((static_cast<unsigned>(n) + static_cast<unsigned>(size) - 1u) / static_cast<unsigned>(size));
}

struct I8Tile {
    int expert;
    int m0, m1;  // rows of A: the tile's first, the expert's end
    int n0;
};

// Raster of one expert's (or the one matrix's) tiles: groups of 16 token
// tiles, so that tiles running together share panels of both operands.
constexpr int kI8GroupM = 16;

struct I8Sched {
    int experts, M, tiles_n, num_tiles;
    const int *off;         // shared memory: experts + 1 clamped offsets
    const int *tile_start;  // shared memory: experts + 1 first tiles
};

template <int BT>
__device__ __forceinline__ I8Tile i8_tile(const I8Sched &s, int t)
{
    I8Tile ti;
    int local = t, rows = s.M;
    ti.expert = 0;
    ti.m0 = 0;
    ti.m1 = s.M;
    if (s.experts) {
        int lo = 0, hi = s.experts - 1;
        while (lo < hi) {  // last expert whose first tile is <= t
            const int mid = (lo + hi + 1) >> 1;
            if (s.tile_start[mid] <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        ti.expert = lo;
        ti.m0 = s.off[lo];
        ti.m1 = s.off[lo + 1];
        rows = ti.m1 - ti.m0;
        local = t - s.tile_start[lo];
    }
    const int tiles_m = i8_tiles(rows, BT);
    const int per_group = kI8GroupM * s.tiles_n;
    const int g = local / per_group;
    const int first = g * kI8GroupM;
    const int in_group = min(tiles_m - first, kI8GroupM);
    const int r = local - g * per_group;
    ti.m0 += (first + r % in_group) * BT;
    ti.n0 = (r / in_group) * kI8Channels;
    return ti;
}

// 3-D tiled load (the experts' matrices): coordinates (k, n, expert).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *map, uint32_t bar, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// Four int8 to four fp16: with its sign bit flipped a byte is q + 128; as the
// low byte of 0x64xx it is the fp16 number 1024 + q + 128, from which 1152 is
// taken off exactly.
__device__ __forceinline__ void widen4(uint32_t q, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = q ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off);
    __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
    lo = *reinterpret_cast<uint32_t *>(&x);
    hi = *reinterpret_cast<uint32_t *>(&y);
}

// One 16-byte unit of a raw row (unit c of row r of a 128-byte-swizzled int8
// tile) to the two units it fills in row r of an fp16 tile.
__device__ __forceinline__ void convert_unit(uint32_t raw, uint32_t conv, int r, int c_raw, int u)
{
    const uint32_t key = static_cast<uint32_t>(r) & 7u;
    uint32_t q[4], h[8];
    ld_shared_v4(raw + r * 128 + ((static_cast<uint32_t>(c_raw) ^ key) << 4), q[0], q[1], q[2], q[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        widen4(q[i], h[2 * i], h[2 * i + 1]);
    st_shared_v4(conv + r * 128 + ((static_cast<uint32_t>(u) ^ key) << 4), h[0], h[1], h[2], h[3]);
    st_shared_v4(conv + r * 128 + ((static_cast<uint32_t>(u + 1) ^ key) << 4), h[4], h[5], h[6], h[7]);
}

template <typename D>
__device__ __forceinline__ void store_scaled(D *p, float v);
template <>
__device__ __forceinline__ void store_scaled<float>(float *p, float v)
{
    *p = v;
}
template <>
__device__ __forceinline__ void store_scaled<__nv_bfloat16>(__nv_bfloat16 *p, float v)
{
    *p = __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ void store_scaled<__half>(__half *p, float v)
{
    *p = __float2half_rn(v);
}

// ---------------------------------------------------------------- kernel

template <int BT, typename D>
__global__ void __launch_bounds__(kI8Threads, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ I8Params p)
{
    using C = I8Cfg<BT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_addr);
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);

    const uint32_t bar_raw_full = base + C::BAR_OFF;
    const uint32_t bar_raw_empty = bar_raw_full + 8 * C::RAW_STAGES;
    const uint32_t bar_conv_full = bar_raw_empty + 8 * C::RAW_STAGES;
    const uint32_t bar_conv_empty = bar_conv_full + 8 * C::CONV_STAGES;
    const uint32_t bar_acc_full = bar_conv_empty + 8 * C::CONV_STAGES;
    const uint32_t bar_acc_empty = bar_acc_full + 16;
    const uint32_t bar_drain = bar_acc_empty + 16;
    const uint32_t bar_inject = bar_drain + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + C::MISC_OFF + 4);
    int *off = reinterpret_cast<int *>(smem + C::MISC_OFF + 16);
    int *tile_start = off + p.experts + 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::RAW_STAGES; ++s) {
            mbar_init(bar_raw_full + 8 * s, 1);
            mbar_init(bar_raw_empty + 8 * s, kI8ConvWarps);
        }
        for (int s = 0; s < C::CONV_STAGES; ++s) {
            mbar_init(bar_conv_full + 8 * s, kI8ConvWarps);
            mbar_init(bar_conv_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_acc_full + 8 * b, 1);
            mbar_init(bar_acc_empty + 8 * b, kEpiWarps);
        }
        mbar_init(bar_drain, 1);
        mbar_init(bar_inject, 1);
        *abort_flag = 0u;
        fence_mbar_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish<1>();
    }
    if (warp == 2 && p.experts) {
        // clamped offsets and the first tile of each expert: a running
        // maximum and a running sum, 32 experts at a time
        int low = 0, tiles = 0;
        for (int e0 = 0; e0 <= p.experts; e0 += 32) {
            const int e = e0 + lane;
            int v = e <= p.experts ? min(max(p.offsets[e], 0), p.M) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o)
                    v = max(v, x);
            }
            v = max(v, low);
            int prev = __shfl_up_sync(0xffffffffu, v, 1);
            if (lane == 0)
                prev = e0 == 0 ? v : low;
            // tiles of expert e - 1, which lies between prev and v
            int n = e <= p.experts ? i8_tiles(v - prev, BT) * p.tiles_n : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, n, o);
                if (lane >= o)
                    n += x;
            }
            n += tiles;
            if (e <= p.experts) {
                off[e] = v;
                tile_start[e] = n;
            }
            low = __shfl_sync(0xffffffffu, v, 31);
            tiles = __shfl_sync(0xffffffffu, n, 31);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;

    Waiter w;
    w.timeout_ns = p.timeout_ns;
    w.abort_flag = abort_flag;
    w.status = p.status;
    w.all_cluster_scope = false;

    I8Sched sched;
    sched.experts = p.experts;
    sched.M = p.M;
    sched.tiles_n = p.tiles_n;
    sched.off = off;
    sched.tile_start = tile_start;
    sched.num_tiles = p.experts ? tile_start[p.experts] : i8_tiles(p.M, BT) * p.tiles_n;
    const int raw_blocks = i8_tiles(p.K, kI8RawK);
    // K past the end is zeros in the raw tiles; a last block of at most 64
    // elements still fills both fp16 stages
    const int conv_blocks = raw_blocks * (kI8RawK / kI8ConvK);

    ProducerTail tail{0, 0, 0u};
    if (warp == 0) {
        if (lane == 0) {
            if (p.inject == kRoleProducer) {
                w.wait(bar_inject, 0u, kRoleProducer | kWaitInjected);
            } else {
                int stage = 0, issued = 0;
                uint32_t phase = 0;
                bool ok = true;
                for (int t = blockIdx.x; ok && t < sched.num_tiles; t += gridDim.x) {
                    const I8Tile ti = i8_tile<BT>(sched, t);
                    for (int kb = 0; kb < raw_blocks; ++kb) {
                        ok = w.wait(bar_raw_empty + 8 * stage, phase ^ 1u, kRoleProducer | kWaitEmpty);
                        if (!ok)
                            break;
                        const uint32_t dst = base + stage * C::RAW_BYTES, bar = bar_raw_full + 8 * stage;
                        mbar_arrive_expect_tx(bar, C::RAW_BYTES);
                        tma_load_3d(dst, &tmB, bar, kb * kI8RawK, ti.n0, ti.expert);
                        tma_load_2d(dst + C::RAW_W, &tmA, bar, kb * kI8RawK, ti.m0);
                        ++issued;
                        if (++stage == C::RAW_STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
                tail = ProducerTail{issued < C::RAW_STAGES ? issued : C::RAW_STAGES, stage, phase};
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            if (p.inject == kRoleMma)
                w.wait(bar_inject, 0u, kRoleMma | kWaitInjected);
            const uint32_t idesc = make_idesc_f16(kI8Channels, BT, 0, 0, 0);
            const OperandPacking pk = operand_packing(0, 3, kI8Channels, kI8ConvK);
            const uint64_t a_desc = make_smem_desc(base + C::CONV_OFF, pk.lbo, pk.sbo, pk.swz);
            const uint64_t b_desc = make_smem_desc(base + C::CONV_OFF + C::CONV_W, pk.lbo, pk.sbo, pk.swz);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = p.inject != kRoleMma;
            for (int t = blockIdx.x; ok && t < sched.num_tiles; t += gridDim.x) {
                ok = w.wait(bar_acc_empty + 8 * acc, acc_phase ^ 1u, kRoleMma | kWaitAccEmpty);
                if (!ok)
                    break;
                tc_fence_after_sync();
                const uint32_t d = tmem_base + static_cast<uint32_t>(acc * C::ACC_STRIDE);
                for (int kb = 0; kb < conv_blocks; ++kb) {
                    ok = w.wait(bar_conv_full + 8 * stage, phase, kRoleMma | kWaitFull);
                    if (!ok)
                        break;
                    tc_fence_after_sync();
                    const uint64_t step = static_cast<uint64_t>((stage * C::CONV_BYTES) >> 4);
#pragma unroll
                    for (int j = 0; j < kI8ConvK / 16; ++j)
                        mma_f16<1>(d, a_desc + step + 2 * j, b_desc + step + 2 * j, idesc, (kb | j) != 0);
                    mma_commit<1>(bar_conv_empty + 8 * stage);
                    if (++stage == C::CONV_STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok)
                    break;
                mma_commit<1>(bar_acc_full + 8 * acc);
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            // every MMA this thread issued has completed before TMEM is freed
            mma_commit<1>(bar_drain);
            w.drain(bar_drain, 0u, 100000000ull);
        }
    } else if (warp >= kI8FirstConvWarp) {
        const int ct = static_cast<int>(threadIdx.x) - 32 * kI8FirstConvWarp;
        constexpr int kThreads = 32 * kI8ConvWarps;
        int rs = 0, cs = 0;
        uint32_t rphase = 0, cphase = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < sched.num_tiles; t += gridDim.x) {
            for (int kb = 0; ok && kb < raw_blocks; ++kb) {
                ok = w.wait(bar_raw_full + 8 * rs, rphase, kRoleConvert | kWaitRawFull);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                const uint32_t rw = base + rs * C::RAW_BYTES, rx = rw + C::RAW_W;
#pragma unroll 1
                for (int h = 0; h < kI8RawK / kI8ConvK; ++h) {
                    ok = w.wait(bar_conv_empty + 8 * cs, cphase ^ 1u, kRoleConvert | kWaitConvEmpty);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok)
                        break;
                    const uint32_t cw = base + C::CONV_OFF + cs * C::CONV_BYTES, cx = cw + C::CONV_W;
                    // neighbouring threads take neighbouring rows of one unit column: no bank conflicts
#pragma unroll
                    for (int i = ct; i < kI8Channels * 4; i += kThreads) {
                        const int c = i / kI8Channels;
                        convert_unit(rw, cw, i % kI8Channels, 4 * h + c, 2 * c);
                    }
#pragma unroll
                    for (int i = ct; i < BT * 4; i += kThreads) {
                        const int c = i / BT;
                        convert_unit(rx, cx, i % BT, 4 * h + c, 2 * c);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar_conv_full + 8 * cs);
                    if (++cs == C::CONV_STAGES) {
                        cs = 0;
                        cphase ^= 1u;
                    }
                }
                if (!ok)
                    break;
                if (lane == 0)
                    mbar_arrive(bar_raw_empty + 8 * rs);
                if (++rs == C::RAW_STAGES) {
                    rs = 0;
                    rphase ^= 1u;
                }
            }
        }
    } else {
        const int q = warp & 3;  // TMEM lane quarter of this warp
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int t = blockIdx.x; t < sched.num_tiles; t += gridDim.x) {
            const I8Tile ti = i8_tile<BT>(sched, t);
            const int n = ti.n0 + 32 * q + lane;
            const bool live = n < p.N;
            const float sn = live ? p.sb[static_cast<long long>(ti.expert) * p.N + n] : 0.0f;
            bool ok = w.wait(bar_acc_full + 8 * acc, acc_phase, kRoleEpilogue | kWaitAccFull);
            if (!__all_sync(0xffffffffu, ok))
                break;
            tc_fence_after_sync();
            const uint32_t src = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(acc * C::ACC_STRIDE);
            const int rows = min(ti.m1 - ti.m0, BT);
            for (int c = 0; c < rows; c += 32) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(src + c, r);
                const float my_sa = c + lane < rows ? p.sa[ti.m0 + c + lane] : 0.0f;
                tmem_ld_wait();
                D *out = static_cast<D *>(p.d) + static_cast<long long>(ti.m0 + c) * p.ldd + n;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float sm = __shfl_sync(0xffffffffu, my_sa, i);
                    if (live && c + i < rows)
                        store_scaled<D>(out + i * p.ldd, __uint_as_float(r[i]) * sm * sn);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_acc_empty + 8 * acc);
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
    }
    __syncwarp();
    __syncthreads();  // every role has returned: the abort flag is final
    if (*abort_flag && warp == 0 && lane == 0)
        drain_producer_tail<C::RAW_STAGES>(tail, bar_raw_full, w);
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc<1>(tmem_base, C::TMEM_COLS);
    }
}

// Zeros for K == 0: the rows of every expert, or all M of them.
template <typename D>
__global__ void int8_zero_kernel(const I8Params p)
{
    long long rows = p.M;
    if (p.experts) {
        rows = 0;
        for (int e = 0; e <= p.experts; ++e)
            rows = max(rows, min(static_cast<long long>(p.offsets[e]), static_cast<long long>(p.M)));
    }
    const long long first = p.experts ? min(max(p.offsets[0], 0), p.M) : 0;
    for (long long i = blockIdx.x; i + first < rows; i += gridDim.x)
        for (int n = threadIdx.x; n < p.N; n += blockDim.x)
            store_scaled<D>(static_cast<D *>(p.d) + (i + first) * p.ldd + n, 0.0f);
}

template <int BT, typename D>
std::atomic<uint64_t> i8_attribute_set[2] = {{0}, {0}};

template <int BT, typename D>
gemm_status_t launch_int8(const CUtensorMap &a, const CUtensorMap &b, const I8Params &p, int sms, cudaStream_t st)
{
    using C = I8Cfg<BT>;
    auto kern = int8_gemm_kernel<BT, D>;
    const int most = C::SMEM_BASE + 2 * 4 * (GEMM_ROUTE_MAX_EXPERTS + 1);
    if (ensure_smem_attribute(kern, most, i8_attribute_set<BT, D>) != cudaSuccess)
        return GEMM_ERR_CUDA;
    const int smem = C::SMEM_BASE + (p.experts ? 2 * 4 * (p.experts + 1) : 0);
    // tiles of the launch, or for experts the most there can be
    const int64_t tiles_m = (static_cast<int64_t>(p.M) + BT - 1) / BT + (p.experts ? std::min(p.experts, p.M) : 0);
    const int grid = static_cast<int>(std::min<int64_t>(tiles_m * p.tiles_n, sms));
    kern<<<grid, kI8Threads, smem, st>>>(a, b, p);
    return host_launched();
}

template <typename D>
gemm_status_t run_int8_typed(const CUtensorMap &a, const CUtensorMap &b, const I8Params &p, int bt, int sms,
                             cudaStream_t st)
{
    switch (bt) {
    case 16: return launch_int8<16, D>(a, b, p, sms, st);
    case 32: return launch_int8<32, D>(a, b, p, sms, st);
    case 64: return launch_int8<64, D>(a, b, p, sms, st);
    case 128: return launch_int8<128, D>(a, b, p, sms, st);
    default: return launch_int8<256, D>(a, b, p, sms, st);
    }
}

// Tokens per tile: the smallest that takes the rows of one expert (on
// average), 256 only where such tiles fill the SMs.
int int8_tile_tokens(int64_t M, int64_t N, int64_t E, int sms)
{
    const int64_t rows = E ? (M + E - 1) / E : M;
    int bt = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
    const int64_t tiles_n = (N + kI8Channels - 1) / kI8Channels;
    while (bt > 128 && (M + bt - 1) / bt * tiles_n < sms)
        bt /= 2;
    return bt;
}

gemm_status_t run_int8(int64_t M, int64_t N, int64_t K, int64_t E, const int32_t *offsets, const int8_t *A, int64_t lda,
                       const float *sa, const int8_t *B, int64_t ldb, int64_t stride_b, const float *sb, void *D,
                       int64_t ldd, int d_type, cudaStream_t st)
{
    if (!valid_size(M) || !valid_size(N) || !valid_size(K) || !valid_type(d_type))
        return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0)
        return GEMM_OK;
    const int od = type_bytes(d_type);
    if (!sa || !sb || !D || ldd < N || !valid_stride(ldd, od) || (E && !offsets))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(D, od) || !aligned_to(sa, 4) || !aligned_to(sb, 4) || !aligned_to(offsets, 4))
        return GEMM_ERR_ALIGNMENT;
    if (K > 0) {
        if (!A || !B || lda < K || ldb < K || !valid_stride(lda, 1) || !valid_stride(ldb, 1))
            return GEMM_ERR_INVALID_ARG;
        if (E > 1 && (stride_b < 0 || !valid_stride(stride_b, 1) || stride_b < (N - 1) * ldb + K))
            return GEMM_ERR_INVALID_ARG;
        if (!aligned_to(A, 16) || !aligned_to(B, 16) || lda % 16 != 0 || ldb % 16 != 0 || (E > 1 && stride_b % 16 != 0))
            return GEMM_ERR_ALIGNMENT;
    }
    const int64_t tiles_n = (N + kI8Channels - 1) / kI8Channels;
    if (tiles_n * ((M + 15) / 16 + (E ? std::min(E, M) : 0)) > kSizeLimit)
        return GEMM_ERR_UNSUPPORTED;
    int dev = 0, sms = 0;
    unsigned int *status = nullptr;
    gemm_status_t s = host_device(&dev, &status, &sms);
    if (s != GEMM_OK)
        return s;
    I8Params p = {};
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.experts = static_cast<int>(E);
    p.offsets = offsets;
    p.tiles_n = static_cast<int>(tiles_n);
    p.sa = sa;
    p.sb = sb;
    p.d = D;
    p.ldd = ldd;
    p.out_type = d_type;
    p.status = status;
    if (K == 0) {
        const int grid = static_cast<int>(std::min<int64_t>(M, 8 * sms));
        if (d_type == GEMM_OUT_F32)
            int8_zero_kernel<float><<<grid, 256, 0, st>>>(p);
        else if (d_type == GEMM_OUT_BF16)
            int8_zero_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p);
        else
            int8_zero_kernel<__half><<<grid, 256, 0, st>>>(p);
        return host_launched();
    }
    int ms = 0;
    p.inject = host_take_injection(&ms);
    p.timeout_ns = static_cast<unsigned long long>(ms > 0 ? ms : 2000) * 1000000ull;
    const int bt = int8_tile_tokens(M, N, E, sms);
    CUtensorMap a, b;
    {
        const uint64_t dims[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(M)};
        const uint64_t strides[1] = {static_cast<uint64_t>(lda)};
        const uint32_t box[2] = {kI8RawK, static_cast<uint32_t>(bt)};
        if ((s = host_encode_tiled(&a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, A, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) !=
            GEMM_OK)
            return s;
    }
    {
        const uint64_t dims[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(E ? E : 1)};
        const uint64_t strides[2] = {static_cast<uint64_t>(ldb), static_cast<uint64_t>(E > 1 ? stride_b : ldb)};
        const uint32_t box[3] = {kI8RawK, kI8Channels, 1};
        if ((s = host_encode_tiled(&b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, B, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) !=
            GEMM_OK)
            return s;
    }
    if (d_type == GEMM_OUT_F32)
        return run_int8_typed<float>(a, b, p, bt, sms, st);
    if (d_type == GEMM_OUT_BF16)
        return run_int8_typed<__nv_bfloat16>(a, b, p, bt, sms, st);
    return run_int8_typed<__half>(a, b, p, bt, sms, st);
}

}  // namespace g300

extern "C" {

gemm_status_t gemm_int8(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, const float *scale_a,
                        const int8_t *B, int64_t ldb, const float *scale_b, void *D, int64_t ldd, gemm_out_t d_type,
                        gemm_stream_t stream)
{
    return g300::run_int8(M, N, K, 0, nullptr, A, lda, scale_a, B, ldb, 0, scale_b, D, ldd, d_type,
                          reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_int8_grouped(int64_t M, int64_t N, int64_t K, int64_t E, const int32_t *offsets, const int8_t *A,
                                int64_t lda, const float *scale_a, const int8_t *B, int64_t ldb, int64_t stride_b,
                                const float *scale_b, void *D, int64_t ldd, gemm_out_t d_type, gemm_stream_t stream)
{
    if (E < 1 || E > GEMM_ROUTE_MAX_EXPERTS)
        return GEMM_ERR_INVALID_ARG;
    return g300::run_int8(M, N, K, E, offsets, A, lda, scale_a, B, ldb, stride_b, scale_b, D, ldd, d_type,
                          reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
