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
// multiply and sum them in fp32 (exact below 2^24). The widened rows of the
// MMA's M side go to Tensor Memory, from where the MMA takes its first operand,
// those of its N side to shared memory: with both in shared memory a 128 x 256
// tile moves 288 bytes of it per MMA cycle (raw writes and reads, fp16 writes,
// MMA reads) where an SM moves 128, which held 8192^3 at 0.48 of the tensor rate.
//
// Two shapes of tile:
//   narrow  128 channels (rows of B) on the M side, 16 to 64 tokens (rows of
//           A) on the N side, or 256 channels and 128 tokens on a CTA pair: few
//           tokens still use whole MMA rows and every weight is read once. Such MMAs are short and the
//           issuing thread, about 1000 cycles for the eight of a stage, is
//           the limit; so two threads issue alternate stages, each into an
//           accumulator of its own, and the epilogue adds the two. For few
//           tiles a cluster of CTAs shares one tile's K (KS > 1): the others
//           leave their fp32 sums in the first CTA's shared memory, which adds
//           them in the order of their ranks.
//   wide    256 tokens on the M side, 256 channels on the N side, CTA pairs
//           (cta_group::2; each CTA widens its 128 tokens and half of the
//           channels): a stage's eight MMAs take 1024 cycles and keep the
//           tensor pipe fed. One accumulator of 256 columns fits beside the
//           widened stages, so what counts is how soon it is empty again: the
//           sixteen converter warps widen the first blocks of the next tile,
//           take the accumulator into registers at one go, and store it while
//           the MMAs run on those blocks.
//
// Warp roles of a CTA:
//   warp 0       TMA producer: raw int8 stages of 128 elements of K;
//   warp 1       TMEM allocator and MMA issuer (pairs: of the even CTA);
//   warp 2       narrow: second MMA issuer; warp 3 completes the warpgroup;
//   warps 4-7    narrow: epilogue;
//   the last 16  converters (wide: and epilogue) in two groups of 8 warps that take alternate
//                stages; a group reads and widens a stage into registers
//                before it waits for room to write it. The warpgroups share
//                the registers out by need (setmaxnreg).
// Every wait is bounded, as in gemm_kernel.cuh, here by the length of K.
//
// Measured on a GB300, operands not in L2, launches one after another (HBM 6.78
// TB/s, bf16 products 1932 TFLOP/s): 8192^3 547 us in a burst of 20 launches
// (2010 TFLOP/s) and 620 us in a long run under the power cap (1770), 4096^3 86
// us (256 wide tiles on 76 pairs: 4 rounds for 3.4), 8192^2 x 2048 167 us (an
// epilogue for each sixteen stages), 64 experts with 512 rows each, N 4096, K
// 2048 335 us; 128 x 16384 x 4096 20.5-21.6 us, 16 x 16384 x 4096 15.7 us (about 0.4
// us a stage on 128 CTAs: the issue of 16-token MMAs and the widening, both
// ahead of the 10 us of HBM traffic), 96 rows over 64 experts 88 us (0.9 of the
// HBM rate). What bounds wide tiles: shared memory, 128 to 160 KB a stage
// (raw writes and reads, fp16 writes, MMA reads) for 1024 MMA cycles.
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

constexpr int kI8Rows = 128;      // rows of the MMA's M side per CTA
constexpr int kI8K = 128;         // elements of K per stage: one 128-byte swizzled int8 row, two fp16 ones
constexpr int kI8GroupWarps = 8;  // converter warps per group
constexpr int kI8GroupThreads = 32 * kI8GroupWarps;
constexpr int kI8FirstEpiWarp = 4;
constexpr int kI8MaxSmem = 232448;

enum : uint32_t {
    kWaitRawFull = 11 << 8,
    kWaitConvEmpty = 12 << 8,
    kWaitSplit = 13 << 8,
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
    int vec;     // rows of D start on multiples of 32 bytes
    int inject;  // test hook: the role that waits on a barrier nothing arrives at (see the epilogue for its own)
    unsigned long long timeout_ns;
    unsigned int *status;
};

// NS: rows of the N side of one MMA (narrow: tokens; wide: 256 channels).
// Tiles of 128 tokens and wide ones are shared by a pair of CTAs. KS: most CTAs sharing one tile's K (1: none do).
template <int NS, int KS, bool WIDE>
struct I8Cfg {
    static constexpr int CG = WIDE || NS == 128 ? 2 : 1;
    static constexpr int TOKENS = WIDE ? 256 : NS, CHANNELS = WIDE ? NS : 128 * CG;  // of a tile
    static constexpr int SIDE = NS / CG;                                        // N-side rows widened by each CTA
    static constexpr int ISSUERS = WIDE ? 1 : 2;
    static constexpr int EPI_WARPS = WIDE ? 0 : 4;  // of their own
    static constexpr int FIRST_CONV_WARP = kI8FirstEpiWarp + EPI_WARPS;
    static constexpr int THREADS = 32 * (FIRST_CONV_WARP + 2 * kI8GroupWarps);
    // TMEM: accumulators (buffers x issuers), then the widened M side, 64 columns a stage
    static constexpr int ACC_STRIDE = NS < 32 ? 32 : NS;  // whole 32-column epilogue reads
    static constexpr int ACC_BUFS = WIDE || NS == 128 ? 1 : 2;
    static constexpr int A_COL0 = ACC_BUFS * ISSUERS * ACC_STRIDE;
    static constexpr int A_COLS = kI8K / 2;
    static constexpr int CONV_FIT = (512 - A_COL0) / A_COLS;
    static constexpr int CONV_MOST = WIDE ? 2 : 4;  // shared memory has room for
    // Both rings have an even number of stages: the two converter groups (and
    // the two issuers) take alternate blocks, so each stage always belongs to
    // the same one. With an odd number a group that runs ahead would wait for
    // the phase after next of a barrier, whose parity is that of the last one.
    static constexpr int CONV_STAGES = CONV_FIT < CONV_MOST ? CONV_FIT : CONV_MOST;
    static constexpr int RAW_M = kI8Rows * kI8K;
    static constexpr int RAW_BYTES = RAW_M + SIDE * kI8K;
    static constexpr int CONV_BYTES = 2 * SIDE * kI8K;  // two tiles of 64 elements of K
    static constexpr int PART_BYTES = (KS - 1) * NS * kI8Rows * 4;
    static constexpr int EPI_BYTES = WIDE ? 2 * kI8GroupWarps * 1024 : 0;  // 8 x 32 fp32 a warp
    static constexpr int FIXED = CONV_STAGES * CONV_BYTES + PART_BYTES + EPI_BYTES + 1024 /* alignment */ +
                                 512 /* barriers */ + 2 * 4 * (GEMM_ROUTE_MAX_EXPERTS + 1);
    static constexpr int RAW_FIT = (kI8MaxSmem - FIXED) / RAW_BYTES;
    static constexpr int RAW_STAGES = RAW_FIT < 8 ? RAW_FIT & ~1 : 8;
    static constexpr int CONV_OFF = RAW_STAGES * RAW_BYTES;
    static constexpr int PART_OFF = CONV_OFF + CONV_STAGES * CONV_BYTES;
    static constexpr int EPI_OFF = PART_OFF + PART_BYTES;
    static constexpr int BAR_OFF = EPI_OFF + EPI_BYTES;
    static constexpr int NUM_BARS = 2 * RAW_STAGES + 2 * CONV_STAGES + 4 + 3;
    static constexpr int MISC_OFF = BAR_OFF + 8 * NUM_BARS;
    static constexpr int TABLE_OFF = MISC_OFF + 16;
    static constexpr int CLUSTER = CG * KS;  // largest cluster
    // 16-byte units of the N side of a stage per converter thread, and how many
    // unit columns apart a thread's units lie
    static constexpr int UNITS = SIDE * 8 < kI8GroupThreads ? 1 : SIDE * 8 / kI8GroupThreads;
    static constexpr int UNIT_STEP = kI8GroupThreads / SIDE;
    // Registers a thread: at launch, and after the warpgroups have shared them
    // out (producer and issuers; epilogue; converters)
    static constexpr int LAUNCH_REGS = WIDE ? 96 : 80;
    static constexpr int ISSUE_REGS = WIDE ? 32 : 48;
    static constexpr int EPI_REGS = 112;
    static constexpr int CONV_REGS = WIDE ? 112 : 80;
    static constexpr int REG_TOTAL = 128 * (ISSUE_REGS + EPI_WARPS / 4 * EPI_REGS + 4 * CONV_REGS);
    static_assert(REG_TOTAL <= THREADS * LAUNCH_REGS && THREADS * LAUNCH_REGS <= 65536,
                  "the shares add up to no more than the block is launched with");
    static_assert((!WIDE || NS == 256) && (CG == 1 || KS == 1), "wide tiles: 256 channels; pairs do not share K");
    static_assert((SIDE & (SIDE - 1)) == 0 && SIDE >= 16 && SIDE <= 128, "unit arithmetic");
    static_assert(8 * NUM_BARS + 16 <= 512, "barriers");
    static_assert(RAW_BYTES % 1024 == 0 && CONV_BYTES % 1024 == 0 && SIDE * kI8K % 1024 == 0,
                  "swizzle atoms start on 1024-byte boundaries");
    static_assert(CONV_STAGES % 2 == 0 && RAW_STAGES % 2 == 0 && CONV_STAGES >= 2 && RAW_STAGES >= 4, "stages");
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

// Raster of one expert's (or the one matrix's) tiles: groups of 8 token
// tiles, so that tiles running together share panels of both operands.
constexpr int kI8GroupM = 8;

struct I8Sched {
    int experts, M, tiles_n, num_tiles;
    const int *off;         // shared memory: experts + 1 clamped offsets
    const int *tile_start;  // shared memory: experts + 1 first tiles
};

template <int BT, int CH>
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
    ti.n0 = (r / in_group) * CH;
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

// Four int8 to four fp16, in the order 0, 2, 1, 3 (both operands take the same
// order of K, so the sum does not see it): with its sign bit flipped a byte is
// q + 128; as the low byte of 0x64xx it is the fp16 number 1024 + q + 128, from
// which 1152 is taken off exactly. One three-input logic operation masks a
// pair of bytes, flips their signs and sets the exponents.
__device__ __forceinline__ void widen4(uint32_t q, uint32_t &lo, uint32_t &hi)
{
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t a, b;  // (q & 0x00ff00ff) ^ 0x64806480
    asm("lop3.b32 %0, %1, 0x00ff00ff, 0x64806480, 0x6a;" : "=r"(a) : "r"(q));
    asm("lop3.b32 %0, %1, 0x00ff00ff, 0x64806480, 0x6a;" : "=r"(b) : "r"(q >> 8));
    __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off);
    __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
    lo = *reinterpret_cast<uint32_t *>(&x);
    hi = *reinterpret_cast<uint32_t *>(&y);
}

// Sixteen int8 to sixteen fp16.
__device__ __forceinline__ void widen16(const uint4 &q, uint32_t *h)
{
    widen4(q.x, h[0], h[1]);
    widen4(q.y, h[2], h[3]);
    widen4(q.z, h[4], h[5]);
    widen4(q.w, h[6], h[7]);
}

// 32 lanes x 32 consecutive 32-bit columns of TMEM from registers.
__device__ __forceinline__ void tmem_st_words(uint32_t taddr, const uint32_t (&v)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
                 "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, "
                 "%31, %32};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
                 "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
                 "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
                 : "memory");
}

// kind::f16 MMA with the first operand in TMEM (row = lane, two fp16 of K per
// 32-bit column; a pair's CTAs each hold their own 128 rows).
template <int CG>
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate)
{
    if constexpr (CG == 1)
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
                     "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
                     "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
                     : "memory");
}

// Changes the registers a thread of this warpgroup from FROM to TO (every warp
// of the warpgroup executes it).
template <int FROM, int TO>
__device__ __forceinline__ void set_regs()
{
    if constexpr (TO < FROM)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TO));
    else if constexpr (TO > FROM)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TO));
}

// Waiter::wait for the many warps of this kernel: a probe that does not find
// the phase complete sleeps in the hardware until it is, or for 20 us, so that
// waiting warps leave the issue slots to the converters.
__device__ __forceinline__ bool probe_asleep(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity), "r"(20000u)
                 : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool probe_asleep_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity), "r"(20000u)
                 : "memory");
    return ok != 0;
}

struct I8Waiter {
    Waiter w;

    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, uint32_t code, bool cluster = false) const
    {
        if (cluster ? probe_asleep_cluster(bar, parity) : probe_asleep(bar, parity))
            return true;
        const uint64_t t0 = globaltimer_ns();
        while (!(cluster ? probe_asleep_cluster(bar, parity) : probe_asleep(bar, parity))) {
            if (*w.abort_flag)
                return false;
            if (globaltimer_ns() - t0 > w.timeout_ns) {
                w.fail(code);
                return false;
            }
        }
        return true;
    }
};

// Keeps a value in a register from here on: what computes it is not moved past.
__device__ __forceinline__ void pin(uint32_t &v) { asm volatile("" : "+r"(v)); }

// Arrive on the even CTA's barrier for what this warp has read from its TMEM:
// tcgen05.wait::ld and the fence before the thread sync order those reads, the
// arrival itself needs no more than the cluster's scope.
__device__ __forceinline__ void mbar_arrive_peer_read(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// Arrive on the even CTA's barrier for a stage this warp has written into its
// own CTA's shared memory and TMEM, which the pair's MMA reads by the even CTA's
// order: a release at the cluster's scope, after every lane's proxy fence. All
// that it has to order lies in this CTA's shared memory (tcgen05.wait::st has
// completed the rest), so the fence is confined to that (8192^3 547 us, as
// without a fence; 843 with a release of all memory, one a warp and stage).
__device__ __forceinline__ void mbar_arrive_peer_written(uint32_t cluster_bar)
{
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;\n\t"
                 "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
                 : "memory");
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
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

// 32 columns of this lane's sums, from one accumulator or the sum of two.
__device__ __forceinline__ void load_sums(uint32_t src0, uint32_t src1, bool both, float (&v)[32])
{
    uint32_t r[32];
    tmem_ld_32x32b_x32(src0, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = __uint_as_float(r[i]);
    if (both) {
        tmem_ld_32x32b_x32(src1, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] += __uint_as_float(r[i]);
    }
}

// Scaled sums of one 32-token block, lane = channel: `out` is the channel's
// column of D at the block's first token, `rows` of which exist. Eight tokens
// at a time: their scales are fetched from the lanes that hold them before the
// first of them is stored.
template <typename D>
__device__ __forceinline__ void store_block(D *out, long long ldd, const float (&v)[32], float sa, float sn, int rows, bool live)
{
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
        if (i >= rows)
            break;
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = v[i + j] * __shfl_sync(0xffffffffu, sa, i + j) * sn;
        if (live) {
            if (i + 8 <= rows) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    store_scaled<D>(out + (i + j) * ldd, x[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i + j < rows)
                        store_scaled<D>(out + (i + j) * ldd, x[j]);
            }
        }
    }
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void store1(void *d, int type, long long at, float v)
{
    if (type == GEMM_OUT_F32)
        static_cast<float *>(d)[at] = v;
    else if (type == GEMM_OUT_BF16)
        static_cast<__nv_bfloat16 *>(d)[at] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(d)[at] = __float2half_rn(v);
}

__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v)
{
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ void st_global_32bytes(void *p, const uint32_t (&v)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Sixteen neighbouring values of a row of D whose address is a multiple of 32 bytes.
__device__ __forceinline__ void store16(void *d, int type, long long at, const float (&x)[16])
{
    uint32_t r[8];
    if (type == GEMM_OUT_F32) {
        float *o = static_cast<float *>(d) + at;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r[i] = __float_as_uint(x[8 * h + i]);
            st_global_32bytes(o + 8 * h, r);
        }
    } else if (type == GEMM_OUT_BF16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            r[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        st_global_32bytes(static_cast<__nv_bfloat16 *>(d) + at, r);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            r[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        st_global_32bytes(static_cast<__half *>(d) + at, r);
    }
}

// Waits for a wide tile's sums and stores one warp's part of them: lane = token
// (quarter q of this CTA's 128), 64 channels from column block `block`. The
// channels' scales are fetched before the wait, and the sums taken into
// registers and the accumulator released before anything is stored. Where rows
// of D start on 32-byte boundaries every lane writes its token's channels in
// whole 32-byte sectors (8192^2 x 2048: 179 us with 16-byte pieces and 201 us
// through shared memory, row by row, which is left to other rows of D). False
// if the wait gave up.
__device__ __forceinline__ bool store_wide_tile(const I8Params &p, const I8Waiter &w, const I8Tile &ti, uint32_t bar_acc_full,
                                                uint32_t acc_phase, uint32_t bar_acc_empty, uint32_t tmem_base, uint32_t stage,
                                                int rank, int q, int block, int lane)
{
    const int row0 = ti.m0 + rank * kI8Rows + 32 * q, n0 = ti.n0 + 64 * block;
    const int rows = ti.m1 - row0;
    const float sa = lane < rows ? p.sa[row0 + lane] : 0.0f;
    const float *sb = p.sb + static_cast<long long>(ti.expert) * p.N;
    const float s0 = n0 + lane < p.N ? sb[n0 + lane] : 0.0f, s1 = n0 + 32 + lane < p.N ? sb[n0 + 32 + lane] : 0.0f;
    const bool ok = w.wait(bar_acc_full, acc_phase, kRoleEpilogue | kWaitAccFull, true);
    if (!__all_sync(0xffffffffu, ok))
        return false;
    tc_fence_after_sync();
    const uint32_t src = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(64 * block);
    uint32_t v[2][32];
    tmem_ld_32x32b_x32(src, v[0]);
    tmem_ld_32x32b_x32(src + 32, v[1]);
    tmem_ld_wait();
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0)
        mbar_arrive_peer_read(mapa_shared(bar_acc_empty, 0));
    if (rows <= 0)
        return true;
    if (p.vec && n0 + 64 <= p.N) {
        st_shared_f32(stage + 4 * lane, s0);
        st_shared_f32(stage + 128 + 4 * lane, s1);
        __syncwarp();
        const long long at = static_cast<long long>(row0 + lane) * p.ldd + n0;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x[16];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t sn[4];
                    ld_shared_v4(stage + 128 * c + 64 * h + 16 * u, sn[0], sn[1], sn[2], sn[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[4 * u + i] = __uint_as_float(v[c][16 * h + 4 * u + i]) * sa * __uint_as_float(sn[i]);
                }
                if (lane < rows)
                    store16(p.d, p.out_type, at + 32 * c + 16 * h, x);
            }
        __syncwarp();
        return true;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        // eight tokens x 32 channels at a time through a swizzled tile, then a
        // row at a time, a channel a lane
        const int n = n0 + 32 * c + lane;
        const float sn = c ? s1 : s0;
#pragma unroll 1
        for (int eight = 0; eight < 4 && 8 * eight < rows; ++eight) {
            const int lc = lane & 7;
            if ((lane >> 3) == eight) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    st_shared_v4(stage + lc * 128 + ((u ^ lc) << 4),
                                 __float_as_uint(__uint_as_float(v[c][4 * u]) * sa),
                                 __float_as_uint(__uint_as_float(v[c][4 * u + 1]) * sa),
                                 __float_as_uint(__uint_as_float(v[c][4 * u + 2]) * sa),
                                 __float_as_uint(__uint_as_float(v[c][4 * u + 3]) * sa));
            }
            __syncwarp();
            const long long at = static_cast<long long>(row0 + 8 * eight) * p.ldd + n;
#pragma unroll
            for (int row = 0; row < 8; ++row) {
                const float x = ld_shared_f32(stage + row * 128 + (((lane >> 2) ^ row) << 4) + 4 * (lane & 3));
                if (8 * eight + row < rows && n < p.N)
                    store1(p.d, p.out_type, at + row * p.ldd, x * sn);
            }
            __syncwarp();
        }
    }
    return true;
}

// ---------------------------------------------------------------- kernel

template <int NS, int KS, bool WIDE>
__global__ void __launch_bounds__(I8Cfg<NS, KS, WIDE>::THREADS, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ I8Params p, const int ks)
{
    using C = I8Cfg<NS, KS, WIDE>;
    constexpr int CG = C::CG;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_addr);
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    // a pair's CTAs, or the CTAs sharing a tile's K
    const int cluster = CG == 2 ? 2 : KS > 1 ? ks : 1;
    const int rank = C::CLUSTER > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int cluster_id = static_cast<int>(blockIdx.x) / cluster, clusters = static_cast<int>(gridDim.x) / cluster;

    const uint32_t bar_raw_full = base + C::BAR_OFF;
    const uint32_t bar_raw_empty = bar_raw_full + 8 * C::RAW_STAGES;
    const uint32_t bar_conv_full = bar_raw_empty + 8 * C::RAW_STAGES;
    const uint32_t bar_conv_empty = bar_conv_full + 8 * C::CONV_STAGES;
    const uint32_t bar_acc_full = bar_conv_empty + 8 * C::CONV_STAGES;
    const uint32_t bar_acc_empty = bar_acc_full + 16;
    const uint32_t bar_drain = bar_acc_empty + 16;
    const uint32_t bar_inject = bar_drain + 8;
    const uint32_t bar_part = bar_inject + 8;  // the other CTAs' sums have arrived (KS > 1)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + C::MISC_OFF + 4);
    int *off = reinterpret_cast<int *>(smem + C::TABLE_OFF);
    int *tile_start = off + p.experts + 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::RAW_STAGES; ++s) {
            mbar_init(bar_raw_full + 8 * s, 1);
            mbar_init(bar_raw_empty + 8 * s, kI8GroupWarps);
        }
        for (int s = 0; s < C::CONV_STAGES; ++s) {
            mbar_init(bar_conv_full + 8 * s, kI8GroupWarps * CG);
            mbar_init(bar_conv_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_acc_full + 8 * b, C::ISSUERS);
            mbar_init(bar_acc_empty + 8 * b, (WIDE ? 2 * kI8GroupWarps : C::EPI_WARPS) * CG);
        }
        mbar_init(bar_drain, C::ISSUERS);
        mbar_init(bar_inject, 1);
        mbar_init(bar_part, KS > 1 && cluster > 1 ? C::EPI_WARPS * (cluster - 1) : 1);
        *abort_flag = 0u;
        fence_mbar_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    if (warp == 1) {
        tmem_alloc<CG>(smem_u32(tmem_slot), 512);
        tmem_relinquish<CG>();
    }
    grid_start();  // what precedes it touches this CTA's own shared memory and TMEM only
    if (warp == kI8FirstEpiWarp && p.experts) {
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
            int n = e <= p.experts ? i8_tiles(v - prev, C::TOKENS) * p.tiles_n : 0;
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
    if constexpr (C::CLUSTER > 1)
        cluster_sync_all();  // the other CTAs' barriers exist before anything signals them
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;

    I8Waiter w;
    w.w.timeout_ns = p.timeout_ns;
    w.w.abort_flag = abort_flag;
    w.w.status = p.status;
    w.w.all_cluster_scope = false;

    I8Sched sched;
    sched.experts = p.experts;
    sched.M = p.M;
    sched.tiles_n = p.tiles_n;
    sched.off = off;
    sched.tile_start = tile_start;
    sched.num_tiles = p.experts ? tile_start[p.experts] : i8_tiles(p.M, C::TOKENS) * p.tiles_n;
    // this CTA's K blocks of a tile (zeros past the end of K)
    const int all_blocks = i8_tiles(p.K, kI8K);
    int kb0 = 0, kb1 = all_blocks;
    if constexpr (KS > 1) {
        kb0 = static_cast<int>(static_cast<long long>(all_blocks) * rank / cluster);
        kb1 = static_cast<int>(static_cast<long long>(all_blocks) * (rank + 1) / cluster);
    }

    ProducerTail tail{0, 0, 0u};
    if (warp < kI8FirstEpiWarp) {
        set_regs<C::LAUNCH_REGS, C::ISSUE_REGS>();
        if (warp == 0 && lane == 0) {
            if (p.inject == kRoleProducer) {
                w.wait(bar_inject, 0u, kRoleProducer | kWaitInjected);
            } else {
                int stage = 0, issued = 0;
                uint32_t phase = 0;
                bool ok = true;
                for (int t = cluster_id; ok && t < sched.num_tiles; t += clusters) {
                    const I8Tile ti = i8_tile<C::TOKENS, C::CHANNELS>(sched, t);
                    // a pair's CTAs take their own halves of both sides
                    const int pair_rank = CG == 2 ? rank : 0;
                    const int m0 = ti.m0 + pair_rank * (WIDE ? kI8Rows : C::SIDE), n0 = ti.n0 + pair_rank * (WIDE ? C::SIDE : kI8Rows);
                    for (int kb = kb0; kb < kb1; ++kb) {
                        ok = w.wait(bar_raw_empty + 8 * stage, phase ^ 1u, kRoleProducer | kWaitEmpty);
                        if (!ok)
                            break;
                        const uint32_t dst = base + stage * C::RAW_BYTES, bar = bar_raw_full + 8 * stage;
                        mbar_arrive_expect_tx(bar, C::RAW_BYTES);
                        tma_load_3d(WIDE ? dst + C::RAW_M : dst, &tmB, bar, kb * kI8K, n0, ti.expert);
                        tma_load_2d(WIDE ? dst : dst + C::RAW_M, &tmA, bar, kb * kI8K, m0);
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
        const int issuer = warp - 1;  // takes every ISSUERS-th stage
        if (issuer >= 0 && issuer < C::ISSUERS && lane == 0 && (CG == 1 || rank == 0)) {
            if (p.inject == kRoleMma)
                w.wait(bar_inject, 0u, kRoleMma | kWaitInjected);
            const uint32_t idesc = make_idesc_f16(CG * kI8Rows, NS, 0, 0, 0);
            const OperandPacking pk = operand_packing(0, 3, C::SIDE, kI8K / 2);
            const uint64_t b_desc = make_smem_desc(base + C::CONV_OFF, pk.lbo, pk.sbo, pk.swz);
            int stage = issuer, acc = 0, skip = issuer;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = p.inject != kRoleMma;
            for (int t = cluster_id; ok && t < sched.num_tiles; t += clusters) {
                ok = w.wait(bar_acc_empty + 8 * acc, acc_phase ^ 1u, kRoleMma | kWaitAccEmpty, CG == 2);
                if (!ok)
                    break;
                tc_fence_after_sync();
                const uint32_t d = tmem_base + static_cast<uint32_t>((acc * C::ISSUERS + issuer) * C::ACC_STRIDE);
                int kb = kb0 + skip;
                uint32_t accumulate = 0;
                for (; kb < kb1; kb += C::ISSUERS) {
                    ok = w.wait(bar_conv_full + 8 * stage, phase, kRoleMma | kWaitFull, CG == 2);
                    if (!ok)
                        break;
                    tc_fence_after_sync();
                    const uint32_t a = tmem_base + static_cast<uint32_t>(C::A_COL0 + stage * C::A_COLS);
                    const uint64_t b = b_desc + static_cast<uint64_t>((stage * C::CONV_BYTES) >> 4);
#pragma unroll
                    for (int j = 0; j < kI8K / 16; ++j) {
                        mma_f16_ta<CG>(d, a + 8 * j, b + (j >> 2) * ((C::SIDE * kI8K) >> 4) + 2 * (j & 3), idesc, accumulate);
                        accumulate = 1;
                    }
                    if constexpr (CG == 2)
                        mma_commit_pair_multicast(bar_conv_empty + 8 * stage);
                    else
                        mma_commit<1>(bar_conv_empty + 8 * stage);
                    if ((stage += C::ISSUERS) >= C::CONV_STAGES) {
                        stage -= C::CONV_STAGES;
                        phase ^= 1u;
                    }
                }
                if (!ok)
                    break;
                skip = kb - kb1;
                if constexpr (CG == 2)
                    mma_commit_pair_multicast(bar_acc_full + 8 * acc);
                else
                    mma_commit<1>(bar_acc_full + 8 * acc);
                if (++acc == C::ACC_BUFS) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            // every MMA this thread issued has completed before TMEM is freed
            mma_commit<CG>(bar_drain);
            w.w.drain(bar_drain, 0u, 100000000ull);
        }
    } else if (warp >= C::FIRST_CONV_WARP) {
        set_regs<C::LAUNCH_REGS, C::CONV_REGS>();
        const int cw = warp - C::FIRST_CONV_WARP;
        const int group = cw / kI8GroupWarps;
        const int ct = (cw % kI8GroupWarps) * 32 + lane;  // thread within the group
        const int q = warp & 3;                           // TMEM lane quarter this warp may write
        const int half = (cw >> 2) & 1;                   // the 64 elements of K of its M-side row
        // This thread's share of a stage: 64 elements of one M-side row, and
        // every 256th 16-byte unit of the N side. Neighbouring threads take
        // neighbouring rows, whose swizzled units lie in distinct banks. A
        // unit's column enters its address by XOR, so that one offset serves
        // all of a thread's units.
        uint32_t w_at = static_cast<uint32_t>((32 * q + lane) * kI8K + (((4 * half) ^ (lane & 7)) << 4));
        const int r = ct % C::SIDE, c0 = ct / C::SIDE;
        uint32_t x_at = static_cast<uint32_t>(C::RAW_M + r * kI8K + ((c0 ^ (r & 7)) << 4));
        // a raw unit fills two fp16 units: the second at the first's offset ^ 16
        uint32_t y_at = static_cast<uint32_t>((c0 >> 2) * (C::SIDE * kI8K) + r * kI8K + (((2 * (c0 & 3)) ^ (r & 7)) << 4));
        pin(w_at);
        pin(x_at);
        pin(y_at);
        const bool has_unit = C::SIDE * 8 >= kI8GroupThreads || ct < C::SIDE * 8;  // fewer units than threads
        const uint32_t conv_full = CG == 2 ? mapa_shared(bar_conv_full, 0) : bar_conv_full;
        // the group's next stage, raw and widened: every second one
        int rs = group % C::RAW_STAGES, cs = group % C::CONV_STAGES;
        uint32_t rphase = 0, cphase = 1;
        int skip = group;  // blocks of the tile before the group's next one
        bool ok = p.inject != kRoleConvert;
        if (!ok)
            w.wait(bar_inject, 0u, kRoleConvert | kWaitInjected);
        // wide: the tile whose sums are still to be stored, and the parity of its accumulator
        int done = -1;
        uint32_t acc_phase = 0;
        const uint32_t epi_stage = base + static_cast<uint32_t>(C::EPI_OFF + (WIDE ? cw * 1024 : 0));
        for (int t = cluster_id; ok && t < sched.num_tiles; t += clusters) {
            int kb = kb0 + skip;
            for (; kb < kb1; kb += 2) {
                ok = w.wait(bar_raw_full + 8 * rs, rphase, kRoleConvert | kWaitRawFull);
                if (!(ok = __all_sync(0xffffffffu, ok)))
                    break;
                const uint32_t raw = base + static_cast<uint32_t>(rs * C::RAW_BYTES);
                uint32_t hw[32], hx[C::UNITS][8];
                {
                    uint4 u[4], x[C::UNITS];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        ld_shared_v4((raw + w_at) ^ static_cast<uint32_t>(i << 4), u[i].x, u[i].y, u[i].z, u[i].w);
#pragma unroll
                    for (int i = 0; i < C::UNITS; ++i)
                        if (has_unit)
                            ld_shared_v4((raw + x_at) ^ static_cast<uint32_t>((i * C::UNIT_STEP) << 4), x[i].x, x[i].y, x[i].z, x[i].w);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        widen16(u[i], hw + 8 * i);
#pragma unroll
                    for (int i = 0; i < C::UNITS; ++i)
                        widen16(x[i], hx[i]);
                    // all of it before the wait for room: only the writes follow it
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        pin(hw[i]);
#pragma unroll
                    for (int i = 0; i < C::UNITS * 8; ++i)
                        pin(hx[i / 8][i % 8]);
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_raw_empty + 8 * rs);
                ok = w.wait(bar_conv_empty + 8 * cs, cphase, kRoleConvert | kWaitConvEmpty, CG == 2);
                if (!(ok = __all_sync(0xffffffffu, ok)))
                    break;
                tc_fence_after_sync();
                tmem_st_words(tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                  static_cast<uint32_t>(C::A_COL0 + cs * C::A_COLS + 32 * half),
                              hw);
                const uint32_t conv = base + static_cast<uint32_t>(C::CONV_OFF + cs * C::CONV_BYTES);
#pragma unroll
                for (int i = 0; i < C::UNITS; ++i)
                    if (has_unit) {
                        const int c = i * C::UNIT_STEP;  // unit columns from the thread's first
                        const uint32_t at = ((conv + y_at) ^ static_cast<uint32_t>((2 * (c & 3)) << 4)) +
                                            static_cast<uint32_t>((c >> 2) * (C::SIDE * kI8K));
                        st_shared_v4(at, hx[i][0], hx[i][1], hx[i][2], hx[i][3]);
                        st_shared_v4(at ^ 16u, hx[i][4], hx[i][5], hx[i][6], hx[i][7]);
                    }
                fence_proxy_async_smem();
                tmem_st_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2)
                        mbar_arrive_peer_written(conv_full + 8 * cs);
                    else
                        mbar_arrive(conv_full + 8 * cs);
                }
                if ((rs += 2) >= C::RAW_STAGES) {
                    rs -= C::RAW_STAGES;
                    rphase ^= 1u;
                }
                if ((cs += 2) >= C::CONV_STAGES) {
                    cs -= C::CONV_STAGES;
                    cphase ^= 1u;
                }
                if (WIDE && done >= 0) {
                    ok = store_wide_tile(p, w, i8_tile<C::TOKENS, C::CHANNELS>(sched, done), bar_acc_full, acc_phase, bar_acc_empty, tmem_base,
                                             epi_stage, rank, q, cw >> 2, lane);
                    done = -1;
                    acc_phase ^= 1u;
                    if (!ok)
                        break;
                }
            }
            skip = kb - kb1;  // 0 or 1 of the next tile's blocks is the other group's
            if (WIDE && ok && done >= 0) {  // a tile without a block of this group
                ok = store_wide_tile(p, w, i8_tile<C::TOKENS, C::CHANNELS>(sched, done), bar_acc_full, acc_phase, bar_acc_empty, tmem_base,
                                     epi_stage, rank, q, cw >> 2, lane);
                acc_phase ^= 1u;
            }
            done = t;
        }
        if (WIDE && ok && done >= 0)
            store_wide_tile(p, w, i8_tile<C::TOKENS, C::CHANNELS>(sched, done), bar_acc_full, acc_phase, bar_acc_empty, tmem_base,
                            epi_stage, rank, q, cw >> 2, lane);
    } else if (!WIDE) {
        set_regs<C::LAUNCH_REGS, C::EPI_REGS>();
        const int q = warp & 3;  // TMEM lane quarter of this warp
        const int blocks = kb1 - kb0;
        int acc = 0;
        uint32_t acc_phase = 0;
        int first = 0;  // narrow: the issuer of the tile's first block
        // the injected epilogue waits, or where CTAs share K keeps its sums from the first CTA, which waits for them
        const bool injected = p.inject == kRoleEpilogue && (cluster == CG || rank > 0);
        if (injected && cluster == CG)
            w.wait(bar_inject, 0u, kRoleEpilogue | kWaitInjected);
        for (int t = cluster_id; !injected && t < sched.num_tiles; t += clusters) {
            const I8Tile ti = i8_tile<C::TOKENS, C::CHANNELS>(sched, t);
            const float *sb = p.sb + static_cast<long long>(ti.expert) * p.N;
            {
                // lane = channel, column = token
                const int n = ti.n0 + (CG == 2 ? rank * kI8Rows : 0) + 32 * q + lane;
                const bool live = n < p.N;
                const float sn = live ? sb[n] : 0.0f;
                const int rows = min(ti.m1 - ti.m0, NS);
                float sa = lane < rows ? p.sa[ti.m0 + lane] : 0.0f;  // of the first 32 tokens
                bool ok = w.wait(bar_acc_full + 8 * acc, acc_phase, kRoleEpilogue | kWaitAccFull, CG == 2);
                if (!__all_sync(0xffffffffu, ok))
                    break;
                tc_fence_after_sync();
                // the issuers' sums; a single block leaves one of them unwritten
                const uint32_t lanes = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                       static_cast<uint32_t>(acc * C::ISSUERS * C::ACC_STRIDE);
                const uint32_t src0 = lanes + static_cast<uint32_t>(blocks > 1 ? 0 : first * C::ACC_STRIDE);
                const uint32_t src1 = lanes + static_cast<uint32_t>(C::ACC_STRIDE);
                first = (first + blocks) & 1;
                if (KS > 1 && rank > 0) {
                    // this CTA's sums to the first CTA, [rank - 1][token][channel]
                    const uint32_t part = mapa_shared(base + C::PART_OFF, 0) +
                                          4u * static_cast<uint32_t>(((rank - 1) * NS) * kI8Rows + 32 * q + lane);
                    for (int c = 0; c < rows; c += 32) {
                        float v[32];
                        load_sums(src0 + c, src1 + c, blocks > 1, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i < rows)
                                st_cluster_f32(part + 4u * static_cast<uint32_t>((c + i) * kI8Rows), v[i]);
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_cluster(mapa_shared(bar_part, 0));
                } else {
                    if (KS > 1 && cluster > 1) {
                        ok = w.wait(bar_part, 0u, kRoleEpilogue | kWaitSplit, true);
                        if (!__all_sync(0xffffffffu, ok))
                            break;
                    }
                    for (int c = 0; c < rows; c += 32) {
                        const int left = rows - c;
                        if (c > 0)
                            sa = lane < left ? p.sa[ti.m0 + c + lane] : 0.0f;
                        float v[32];
                        load_sums(src0 + c, src1 + c, blocks > 1, v);
                        if constexpr (KS > 1) {
                            const float *part = reinterpret_cast<const float *>(smem + C::PART_OFF) + c * kI8Rows + 32 * q + lane;
                            for (int k = 1; k < cluster; ++k, part += NS * kI8Rows) {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (i < left)
                                        v[i] += part[i * kI8Rows];
                            }
                        }
                        const long long at = static_cast<long long>(ti.m0 + c) * p.ldd + n;
                        if (p.out_type == GEMM_OUT_F32)
                            store_block(static_cast<float *>(p.d) + at, p.ldd, v, sa, sn, left, live);
                        else if (p.out_type == GEMM_OUT_BF16)
                            store_block(static_cast<__nv_bfloat16 *>(p.d) + at, p.ldd, v, sa, sn, left, live);
                        else
                            store_block(static_cast<__half *>(p.d) + at, p.ldd, v, sa, sn, left, live);
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2)
                        mbar_arrive_peer_read(mapa_shared(bar_acc_empty + 8 * acc, 0));
                    else
                        mbar_arrive(bar_acc_empty + 8 * acc);
                }
            }
            if (++acc == C::ACC_BUFS) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
    }
    __syncwarp();
    __syncthreads();  // every role has returned: the abort flag is final
    if (*abort_flag && warp == 0 && lane == 0)
        drain_producer_tail<C::RAW_STAGES>(tail, bar_raw_full, w.w);
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (C::CLUSTER > 1)
        cluster_sync_all();  // no CTA exits while another may still write into it
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc<CG>(tmem_base, 512);
    }
}

// ---------------------------------------------------------------- few tokens
//
// Up to MT tokens against every channel, for which latency counts: a block
// takes a few channels and its eight warps slices of K, so that all of a
// block's weights are asked for at once (16 bytes a lane and channel), and
// dp4a sums them in 32-bit integers, exactly for K < 2^17. No tile to fill, no
// stages: the weights are read once, the tokens' rows come from L2. One token
// against 4096 x 4096 weights takes 4.2 us (4.0 TB/s, 2 us of it latency),
// against 16384 x 4096 11.7 us (5.8 TB/s).

constexpr int kFewWarps = 8;
constexpr int64_t kFewMaxK = (1 << 17) - 1;

// Bytes k .. k+15 of a row of K: zeros past its end, which is not read past.
// STREAM: read once, so not kept in L1.
template <bool STREAM>
__device__ __forceinline__ int4 load_row16(const int8_t *row, int k, int K)
{
    if (k + 16 <= K) {
        int4 v;
        if constexpr (STREAM)
            asm volatile("ld.global.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "l"(row + k));
        else
            v = *reinterpret_cast<const int4 *>(row + k);
        return v;
    }
    int4 v = make_int4(0, 0, 0, 0);
    int8_t *b = reinterpret_cast<int8_t *>(&v);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (k + i < K)
            b[i] = row[k + i];
    return v;
}

template <int MT, int ROWS>
__global__ void __launch_bounds__(32 * kFewWarps)
    int8_few_kernel(const int8_t *A, long long lda, const int8_t *B, long long ldb, const I8Params p)
{
    __shared__ int part[kFewWarps][ROWS * MT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = blockIdx.x * ROWS;
    grid_start();
    int acc[ROWS][MT] = {};
    for (int k = warp * 512 + lane * 16; k < p.K; k += kFewWarps * 512) {
        int4 w[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)  // rows past the last repeat it; their sums are not stored
            w[r] = load_row16<true>(B + static_cast<long long>(min(n0 + r, p.N - 1)) * ldb, k, p.K);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int4 a = load_row16<false>(A + static_cast<long long>(min(m, p.M - 1)) * lda, k, p.K);
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                acc[r][m] = __dp4a(w[r].x, a.x, __dp4a(w[r].y, a.y, __dp4a(w[r].z, a.z, __dp4a(w[r].w, a.w, acc[r][m]))));
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int s = __reduce_add_sync(0xffffffffu, acc[r][m]);
            if (lane == 0)
                part[warp][m * ROWS + r] = s;
        }
    __syncthreads();
    const int m = threadIdx.x / ROWS, n = n0 + threadIdx.x % ROWS;
    if (threadIdx.x < ROWS * MT && m < p.M && n < p.N) {
        int s = 0;
#pragma unroll
        for (int i = 0; i < kFewWarps; ++i)
            s += part[i][threadIdx.x];
        store1(p.d, p.out_type, m * p.ldd + n, static_cast<float>(s) * p.sa[m] * p.sb[n]);
    }
}

// ROWS: channels per block, eight for one token and four for more, whose sums
// would otherwise take the registers of half the blocks.
template <int MT, int ROWS = MT == 1 ? 8 : 4>
gemm_status_t launch_few(const int8_t *A, int64_t lda, const int8_t *B, int64_t ldb, const I8Params &p, cudaStream_t st)
{
    const unsigned grid = (static_cast<unsigned>(p.N) + ROWS - 1) / ROWS;
    return host_launch(int8_few_kernel<MT, ROWS>, grid, 32 * kFewWarps, 0, st, 0, A, static_cast<long long>(lda), B,
                       static_cast<long long>(ldb), p);
}

// Zeros for K == 0: the rows of every expert, or all M of them.
template <typename D>
__global__ void int8_zero_kernel(const I8Params p)
{
    grid_start();
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

template <int NS, int KS, bool WIDE>
std::atomic<uint64_t> i8_attribute_set[2] = {{0}, {0}};

// Launches tiles of 128 channels x NS tokens, `ks` CTAs sharing a tile's K (1
// unless the kernel is built for it and every tile has a cluster of its own),
// or wide tiles.
template <int NS, int KS, bool WIDE>
gemm_status_t launch_int8(const CUtensorMap &a, const CUtensorMap &b, const I8Params &p, int ks, int sms, cudaStream_t st)
{
    using C = I8Cfg<NS, KS, WIDE>;
    auto kern = int8_gemm_kernel<NS, KS, WIDE>;
    constexpr int kBase = C::TABLE_OFF + 1024;
    if (ensure_smem_attribute(kern, kBase + 2 * 4 * (GEMM_ROUTE_MAX_EXPERTS + 1), i8_attribute_set<NS, KS, WIDE>) != cudaSuccess)
        return GEMM_ERR_CUDA;
    // the register shares were added up for this many registers at launch
    static const bool regs_ok = [&] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, kern) == cudaSuccess && at.numRegs * C::THREADS >= C::REG_TOTAL &&
               at.numRegs <= C::LAUNCH_REGS;
    }();
    if (!regs_ok)
        return GEMM_ERR_UNSUPPORTED;
    // tiles of the launch, or for experts the most there can be
    const int64_t tiles_m = (static_cast<int64_t>(p.M) + C::TOKENS - 1) / C::TOKENS + (p.experts ? std::min(p.experts, p.M) : 0);
    const int64_t tiles = tiles_m * p.tiles_n;
    const int cluster = C::CG * ks;
    const unsigned grid = static_cast<unsigned>(KS > 1 ? tiles * cluster : std::min<int64_t>(tiles, sms / cluster) * cluster);
    return host_launch(kern, grid, C::THREADS, kBase + (p.experts ? 2 * 4 * (p.experts + 1) : 0), st,
                       C::CLUSTER > 1 ? static_cast<unsigned>(cluster) : 0u, a, b, p, ks);
}

// How a product is cut: wide tiles, or narrow ones of `ns` tokens with `ks`
// CTAs sharing a tile's K.
struct I8Plan {
    bool wide;
    int ns, ks;
    int tokens() const { return wide ? 256 : ns; }
    int channels() const { return wide || ns == 128 ? 256 : 128; }
    int box_tokens() const { return wide ? 128 : ns == 128 ? 64 : ns; }  // tokens one CTA loads
};

// CTAs that may share a tile's K: doubled while all tiles still run at once and
// each CTA keeps some blocks.
int int8_shares(int64_t tiles, int64_t blocks, int most, int sms)
{
    int ks = 1;
    while (ks < most && tiles * ks * 2 <= sms && blocks >= 4 * ks)
        ks *= 2;
    return ks;
}

I8Plan int8_plan(int64_t M, int64_t N, int64_t K, int64_t E, int sms)
{
    const int64_t rows = E ? (M + E - 1) / E : M;  // of one matrix, on average
    const int64_t blocks = (K + kI8K - 1) / kI8K;
    auto tiles = [&](int64_t tokens, int64_t channels) { return (M + tokens - 1) / tokens * ((N + channels - 1) / channels); };
    if (rows <= 64) {
        I8Plan pl = {false, rows <= 16 ? 16 : rows <= 32 ? 32 : 64, 1};
        if (E == 0)
            pl.ks = int8_shares(tiles(pl.ns, 128), blocks, pl.ns == 16 ? 8 : pl.ns == 32 ? 4 : 2, sms);
        return pl;
    }
    if (E)
        return {rows > 128 && N > 128, 128, 1};
    // One matrix and more tokens: the tile whose rounds of the grid take least.
    // A block of K takes a CTA 0.43 us on 64 x 128 tiles, 0.51 on pairs of 128 x
    // 256 and 0.66 on wide ones (64, 128 and 768 tokens, 4096 elements of K);
    // wide tiles are far ahead for each product, but a few of them leave most
    // of the SMs idle (100 tokens, 4096 x 4096: 18.0 us on pairs).
    struct Choice {
        I8Plan pl;
        int64_t cost;
    };
    const int ks = int8_shares(tiles(64, 128), blocks, 2, sms);
    auto rounds = [](int64_t n, int64_t units) { return (n + units - 1) / units; };
    const Choice choices[3] = {{{true, 256, 1}, 66 * blocks * rounds(tiles(256, 256), sms / 2)},
                               {{false, 128, 1}, 51 * blocks * rounds(tiles(128, 256), sms / 2)},
                               {{false, 64, ks}, 43 * ((blocks + ks - 1) / ks) * rounds(tiles(64, 128) * ks, sms)}};
    const Choice *best = &choices[0];
    for (const Choice &c : choices)
        if (c.cost < best->cost)
            best = &c;
    return best->pl;
}

// Few tokens, where integers beat tiles, whose work hardly grows with the
// tokens (measured us, integers and tiles: 4096 x 4096 weights with 1, 2, 4
// and 8 tokens 4.2, 5.2, 6.0 and 11.9 against 9.8; 16384 x 4096 11.7, 15.4,
// 19.9 and 27.7 against 15.5; 1024 x 1024 with 8 tokens 2.9 against 5.8).
bool int8_few(int64_t M, int64_t N, int64_t K, int64_t E)
{
    return E == 0 && K <= kFewMaxK &&
           (M <= 2 || (M <= 4 && N * K <= int64_t(1) << 25) || (M <= 8 && N * K <= int64_t(3) << 22));
}

// How long a wait may take: a role may wait for another to walk all of a tile's
// K, for which a block has 10 us (0.4 to 0.7 measured), and 2 s beside it.
int int8_wait_ms(int64_t K, const I8Plan &pl)
{
    return static_cast<int>(2000 + (K / kI8K + 1) / pl.ks / 100);
}

gemm_status_t launch_int8_plan(const CUtensorMap &a, const CUtensorMap &b, const I8Params &p, const I8Plan &pl, int sms,
                               cudaStream_t st)
{
    if (pl.wide)
        return launch_int8<256, 1, true>(a, b, p, 1, sms, st);
    switch (pl.ns) {
    case 16: return pl.ks > 1 ? launch_int8<16, 8, false>(a, b, p, pl.ks, sms, st) : launch_int8<16, 1, false>(a, b, p, 1, sms, st);
    case 32: return pl.ks > 1 ? launch_int8<32, 4, false>(a, b, p, pl.ks, sms, st) : launch_int8<32, 1, false>(a, b, p, 1, sms, st);
    case 64: return pl.ks > 1 ? launch_int8<64, 2, false>(a, b, p, pl.ks, sms, st) : launch_int8<64, 1, false>(a, b, p, 1, sms, st);
    default: return launch_int8<128, 1, false>(a, b, p, 1, sms, st);
    }
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
        // by division: the product of two accepted numbers may pass 64 bits
        if (E > 1 && (stride_b < K || !valid_stride(stride_b, 1) || (N > 1 && (stride_b - K) / (N - 1) < ldb)))
            return GEMM_ERR_INVALID_ARG;
        if (!aligned_to(A, 16) || !aligned_to(B, 16) || lda % 16 != 0 || ldb % 16 != 0 || (E > 1 && stride_b % 16 != 0))
            return GEMM_ERR_ALIGNMENT;
    }
    if (!countable(M) || !countable(N) || !countable(K))
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
    p.sa = sa;
    p.sb = sb;
    p.d = D;
    p.ldd = ldd;
    p.out_type = d_type;
    p.vec = aligned_to(D, 32) && ldd * od % 32 == 0;
    p.status = status;
    if (K == 0) {
        const int grid = static_cast<int>(std::min<int64_t>(M, 8 * sms));
        return host_launch(d_type == GEMM_OUT_F32    ? int8_zero_kernel<float>
                           : d_type == GEMM_OUT_BF16 ? int8_zero_kernel<__nv_bfloat16>
                                                     : int8_zero_kernel<__half>,
                           static_cast<unsigned>(grid), 256, 0, st, 0, p);
    }
    if (int8_few(M, N, K, E))
        return M == 1   ? launch_few<1>(A, lda, B, ldb, p, st)
               : M == 2 ? launch_few<2>(A, lda, B, ldb, p, st)
               : M <= 4 ? launch_few<4>(A, lda, B, ldb, p, st)
                        : launch_few<8>(A, lda, B, ldb, p, st);
    const I8Plan pl = int8_plan(M, N, K, E, sms);
    int ms = 0;
    p.inject = host_take_injection(&ms);
    p.timeout_ns = static_cast<unsigned long long>(ms > 0 ? ms : int8_wait_ms(K, pl)) * 1000000ull;
    const int64_t tiles_n = (N + pl.channels() - 1) / pl.channels();
    if (tiles_n * ((M + pl.tokens() - 1) / pl.tokens() + (E ? std::min(E, M) : 0)) > kSizeLimit)
        return GEMM_ERR_UNSUPPORTED;
    p.tiles_n = static_cast<int>(tiles_n);
    CUtensorMap a, b;
    {
        const uint64_t dims[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(M)};
        const uint64_t strides[1] = {static_cast<uint64_t>(lda)};
        const uint32_t box[2] = {kI8K, static_cast<uint32_t>(pl.box_tokens())};
        if ((s = host_encode_tiled(&a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, A, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) !=
            GEMM_OK)
            return s;
    }
    {
        const uint64_t dims[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(E ? E : 1)};
        const uint64_t strides[2] = {static_cast<uint64_t>(ldb), static_cast<uint64_t>(E > 1 ? stride_b : ldb)};
        const uint32_t box[3] = {kI8K, 128, 1};
        if ((s = host_encode_tiled(&b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, B, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) !=
            GEMM_OK)
            return s;
    }
    return launch_int8_plan(a, b, p, pl, sms, st);
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

gemm_status_t gemm_debug_int8_plan(int64_t M, int64_t N, int64_t K, int64_t E, int sms, int32_t *out)
{
    using namespace g300;
    if (!out || sms <= 0 || M < 1 || N < 1 || K < 1 || E < 0 || E > GEMM_ROUTE_MAX_EXPERTS)
        return GEMM_ERR_INVALID_ARG;
    if (!countable(M) || !countable(N) || !countable(K))
        return GEMM_ERR_UNSUPPORTED;
    const bool few = int8_few(M, N, K, E);
    const I8Plan pl = int8_plan(M, N, K, E, sms);
    out[0] = few ? 0 : pl.wide ? 2 : 1;
    out[1] = few ? static_cast<int32_t>(M) : pl.tokens();
    out[2] = few ? 0 : pl.channels();
    out[3] = few ? 0 : pl.ks;
    out[4] = few ? 0 : int8_wait_ms(K, pl);
    return GEMM_OK;
}

}  // extern "C"
