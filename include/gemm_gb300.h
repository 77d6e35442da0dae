/*
 * gemm_gb300.h -- C ABI of the GB300 (sm_103a) tcgen05 GEMM library.
 *
 * The library computes, for fp16 or bf16 inputs with fp32 accumulation,
 *
 *     D = alpha * A * B + beta * C
 *
 * The product is the tensor-core operation D = A.B + C that the pages build
 * on ("Tensor Cores, layouts, and swizzling", opening section; "06 Blackwell
 * Tensor Core - tcgen05 MMA", "Overview" and the K-step walk-through: the
 * first K step writes the accumulator, later steps add to it). alpha and
 * beta follow BLAS: beta == 0 never reads C.
 *
 * Operand layouts ("LBO, SBO and SWZ for a tcgen05 tile", section 1:
 * K-major and MN-major operands):
 *   A is logical M x K.   GEMM_K_MAJOR: A[m*lda + k]  GEMM_MN_MAJOR: A[k*lda + m]
 *   B is logical K x N.   GEMM_K_MAJOR: B[n*ldb + k]  GEMM_MN_MAJOR: B[k*ldb + n]
 *   C and D are row-major M x N: C[m*ldc + n], D[m*ldd + n]; C has D's type.
 *
 * Ownership: every pointer is a device pointer owned by the caller; the
 * library allocates no device memory on any call. Calls are asynchronous
 * on `stream` (a cudaStream_t; NULL is the legacy default stream). A call
 * that fails validation returns its error at once and enqueues nothing.
 *
 * Requirements (TMA rules, "Tensor Cores, layouts, and swizzling", TMA
 * section: global strides are multiples of 16 bytes and below 2^40):
 *   - A, B, C, D 16-byte aligned; lda, ldb multiples of 8 elements; ldc and
 *     ldd multiples of 16 bytes of the output type;
 *   - M, N, K >= 0, each below 2^31; leading dimensions at least the
 *     stored row length;
 *   - M == 0 or N == 0: nothing to do (GEMM_OK). K == 0: D = beta * C.
 *   - C == D (in place) is allowed; C may be NULL when beta == 0.
 * Violations return GEMM_ERR_INVALID_ARG or GEMM_ERR_ALIGNMENT.
 *
 * Device-side errors: every wait inside the kernels is bounded. A wait that
 * runs out records a code in a device status word and the kernel returns
 * early; gemm_last_device_status() reads (and clears) that word.
 */
#ifndef GEMM_GB300_H
#define GEMM_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;                  /* cudaStream_t is struct CUstream_st* */
typedef struct CUstream_st *gemm_stream_t;

typedef enum {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_ARG = 1,        /* bad size, pointer, enum or option */
    GEMM_ERR_ALIGNMENT = 2,          /* pointer or leading dimension breaks a TMA rule */
    GEMM_ERR_UNSUPPORTED = 3,        /* valid request no compiled kernel variant implements */
    GEMM_ERR_CUDA = 4,               /* a CUDA runtime/driver call failed */
    GEMM_ERR_TIMEOUT = 5             /* a bounded device wait ran out */
} gemm_status_t;

typedef enum { GEMM_K_MAJOR = 0, GEMM_MN_MAJOR = 1 } gemm_major_t;

typedef enum { GEMM_OUT_F32 = 0, GEMM_OUT_BF16 = 1, GEMM_OUT_F16 = 2 } gemm_out_t;

/* Shared-memory swizzle of an operand tile ("Swizzling explained properly",
 * "32B, 64B and 128B swizzles"; raw descriptor codes on the LBO/SBO page,
 * section 4). GEMM_SWIZZLE_AUTO lets the library choose (SW128);
 * GEMM_SWIZZLE_NONE stores plain 8-row x 16-byte core matrices (descriptor
 * code 0, LBO and SBO alone define the layout). GEMM_SWIZZLE_128B_ATOM32 is
 * the page's "128-byte mode with 32-byte atomicity" (descriptor code 1):
 * 128-byte rows whose 32-byte units are XORed with the row index mod 4
 * (Swizzle<2,5,2>, written by TMA's 128B_ATOM_32B mode), read as an MN-major
 * operand with K rows in bands of 4. It is the layout of MN-major TF32
 * operands (gemm_ex in_type 2, the default there); 16- and 8-bit operands
 * refuse it with GEMM_ERR_UNSUPPORTED, because kind::f16 and kind::f8f6f4
 * read such operands as zeros on GB300 (measured). */
typedef enum {
    GEMM_SWIZZLE_AUTO = 0,
    GEMM_SWIZZLE_32B = 1,
    GEMM_SWIZZLE_64B = 2,
    GEMM_SWIZZLE_128B = 3,
    GEMM_SWIZZLE_NONE = 4,
    GEMM_SWIZZLE_128B_ATOM32 = 5
} gemm_swizzle_t;

/*
 * Optional tuning/testing knobs (pass NULL for defaults). Every field 0
 * means "library default".
 *   cta_group     1: one CTA per 128-row tile (tcgen05.mma.cta_group::1);
 *                 2: CTA pairs own 256-row tiles (cta_group::2).
 *   tile_m        accumulator rows per CTA: 128, or 64 (cta_group::1 only:
 *                 tcgen05.mma M = 64 with the TMEM accumulator in Layout F,
 *                 "06 Blackwell Tensor Core - tcgen05 MMA", cta_group::1
 *                 M = 64; default for M <= 64 with 16-bit operands), or 32
 *                 (the weight-stationary tcgen05.mma.ws with M = 32; 16-bit
 *                 operands, single problems, tile_n 256), or 256
 *                 (cta_group::1 only: two M = 128 MMAs per K slice share
 *                 each B slice, their accumulators filling the 512 TMEM
 *                 columns; 16-bit operands, single problems, tile_n 256 or
 *                 224; the epilogue of a tile does not overlap the next
 *                 tile's MMAs; by default 256-wide ones run in pairs of CTAs
 *                 that share B, see multicast_b, and the library takes 224
 *                 where that needs fewer rounds of the grid).
 *   tile_n        MMA N per tile: 64, 128 or 256 (cta_group::2: 128 or 256;
 *                 tile_m 256: 224 or 256).
 *   block_k       K elements per pipeline stage: 32, 64 or 128 where built.
 *   swizzle_a/b   operand swizzle (gemm_swizzle_t).
 *   epilogue_swizzle  1 (default) stages output tiles in SW128 layout;
 *                 -1 stages them unswizzled (bank-conflict ablation).
 *   max_ctas      cap on resident CTAs of the persistent grid.
 *   group_m       tile-raster group height in tiles (L2 reuse).
 *   timeout_ms    bound on each device wait (default 2000 ms).
 *   flags         tuning switches. CTA pairs signal stage and accumulator
 *                 releases to both CTAs with one multicast tcgen05.commit;
 *                 bit 0 instead forwards them from the even CTA with remote
 *                 mbarrier arrives (ablation), bit 1 makes every wait
 *                 acquire at cluster scope (ablation). Bit 2 starts each
 *                 tile's K loop at a per-CTA offset so that CTAs sharing an
 *                 operand panel read different parts of it at a time; with
 *                 flags 0 the library sets it for single problems of at most
 *                 one wave of tiles and at least 16 K blocks (HBM-bound
 *                 shapes such as 16384 x 128 x 8192).
 *                 Bit 3 gives the operand loads an L2 evict_last policy and
 *                 the C loads and D stores evict_first (ablation; no
 *                 measured effect at 4096^3 or 8192^3). Bit 4 (single
 *                 problems with 128-row tiles) reads C from global memory
 *                 straight into the epilogue's registers instead of staging
 *                 it in shared memory by TMA (ablation: 1 % slower at 8192^3).
 *                 Bit 5 splits each stage's loads between two producer
 *                 warps, one for the A boxes (and A scale atoms), one for
 *                 the B boxes (and B scale atoms); NVFP4 kernels, which have
 *                 no room for the second warp, ignore it (ablation: no
 *                 measured effect, the loads are bound by L2 delivery, not
 *                 by the issuing thread). Bit 6 (single problems, 128- and
 *                 256-row tiles) writes D from the epilogue's registers with
 *                 16-byte stores, and reads C into them, instead of staging
 *                 chunks in shared memory for TMA (ablation: equal or up to
 *                 5 % slower at 4096^3 and 8192^3).
 *   stats         diagnostics: NULL, or device memory of 16 uint64 per CTA
 *                 of the grid (at least 16 * number of SMs), where each CTA
 *                 writes cycles its roles spent waiting (slots 0-1 producer,
 *                 2-4 and 8-9 MMA issuer, 5-7 and 10-12 first epilogue warp:
 *                 10-11 stream-K flag waits and partial-sum gathers, 12 the
 *                 cycles after its last accumulator became ready; 13 the
 *                 scale copier of the block-scaled kinds, 14 the MMA issuer
 *                 waiting for a stage's scales).
 *   stream_k      K-split scheduling of single (not grouped) problems with
 *                 128-row tiles, so that a last, partly filled wave of tiles
 *                 does not leave SMs idle: the tiles of whole waves run one
 *                 per cluster as usual, and the K blocks of the remaining
 *                 tiles (the ragged wave plus one full wave, or every tile
 *                 when there are fewer tiles than two waves) are divided
 *                 evenly among all clusters. A cluster that holds the first
 *                 K block of a split tile adds the others' fp32 partial sums
 *                 (left in `workspace`) and writes the tile; the result
 *                 differs from the unsplit one only by summation order.
 *                 The pages have no counterpart; it is a scheduling service
 *                 of this library.
 *                   0 (default) auto: split when `workspace` is given and a
 *                     ragged last wave follows 2 to 7 full waves;
 *                  -1 never; 1 always the split above; 2 split every tile;
 *                   3 split only the tiles of the ragged last wave.
 *                 A split needs at least as many K blocks in the split tiles
 *                 as clusters in the grid, else the launch runs unsplit.
 *   workspace / workspace_bytes  device memory for stream_k (NULL: no
 *                 split): at least gemm_streamk_workspace_size() bytes,
 *                 256-byte aligned, set to zero once before its first use
 *                 (the library leaves it reusable: each launch tags its
 *                 flags with a new value). Calls that may run at the same
 *                 time, on different streams, need different workspaces.
 *   mma_ws        weight-stationary MMA (tcgen05.mma.ws, "How cta_group Sets
 *                 the Operation Scope": one of the choices that fix the
 *                 accumulator layout): 0 the library chooses, 1 use it,
 *                 -1 do not. It serves tiles of 32 or 64 rows of single
 *                 problems with 16-bit operands on one CTA (tile_n 128 or 256
 *                 for 64 rows, 256 for 32); its accumulator is spread over
 *                 the four TMEM lane quarters by column parts, so all four
 *                 epilogue warps store full 32-row chunks. Other tiles with
 *                 mma_ws 1 return GEMM_ERR_UNSUPPORTED.
 *   multicast_b   single-CTA (cta_group::1) tiles 256 wide (128 or 256 rows),
 *                 or 224 wide with 256 rows and K-major B,
 *                 run in clusters of two CTAs on vertically adjacent tiles
 *                 that share their B panel: each CTA loads half of every B
 *                 stage and TMA multicasts it into both CTAs' shared memory,
 *                 so each CTA reads half as many B bytes from L2; each CTA's
 *                 MMA completion releases the stage in both. 0 the library
 *                 chooses (256 x 256 tiles of more than 256 rows in all; 128-row
 *                 tiles when B is MN-major or A and B overflow L2), 1 use it,
 *                 -1 do not; other tiles with 1 return GEMM_ERR_UNSUPPORTED.
 *                 Multicast stays within this GPU's memory (the operands of
 *                 one call).
 */
typedef struct {
    int cta_group;
    int tile_m;
    int tile_n;
    int block_k;
    int swizzle_a;
    int swizzle_b;
    int epilogue_swizzle;
    int max_ctas;
    int group_m;
    int timeout_ms;
    int flags;
    unsigned long long *stats;
    int stream_k;
    void *workspace;
    size_t workspace_bytes;
    int mma_ws;
    int multicast_b;
} gemm_options_t;

/* Bytes of stream-K workspace for any single GEMM on the current device:
 * one 4 x uint32 flag row and one 256 x 256 fp32 partial-sum slot per SM
 * (the largest tile; 128-row tiles use half of each slot).
 * 0 if the device cannot be queried. */
size_t gemm_streamk_workspace_size(void);

/* One problem of a grouped call. All share the call's majors, types,
 * alpha and beta; each has its own sizes, pointers and leading dims. */
typedef struct {
    int64_t M, N, K;
    const void *A;
    const void *B;
    const void *C;
    void *D;
    int64_t lda, ldb, ldc, ldd;
} gemm_problem_t;

/*
 * gemm_bf16 / gemm_f16: one GEMM, inputs bf16 / fp16, fp32 accumulation,
 * output d_type. Tiles of 128 x tile_n (256 x tile_n for CTA pairs) are
 * dealt round-robin to a persistent grid of one CTA per SM; operands reach
 * shared memory by TMA in swizzled layouts, tcgen05.mma accumulates in
 * Tensor Memory, and a warp-specialised epilogue applies alpha/beta and
 * stores D by TMA.
 */
gemm_status_t gemm_bf16(int64_t M, int64_t N, int64_t K,
                        const void *A, gemm_major_t a_major, int64_t lda,
                        const void *B, gemm_major_t b_major, int64_t ldb,
                        const void *C, int64_t ldc,
                        void *D, int64_t ldd, gemm_out_t d_type,
                        float alpha, float beta, gemm_stream_t stream);

gemm_status_t gemm_f16(int64_t M, int64_t N, int64_t K,
                       const void *A, gemm_major_t a_major, int64_t lda,
                       const void *B, gemm_major_t b_major, int64_t ldb,
                       const void *C, int64_t ldc,
                       void *D, int64_t ldd, gemm_out_t d_type,
                       float alpha, float beta, gemm_stream_t stream);

/* The same with explicit options (opts may be NULL). in_type: 0 fp16, 1 bf16,
 * 2 TF32: A and B hold fp32 words (leading dimensions in elements, multiples
 * of 4) and tcgen05 kind::tf32 multiplies their TF32 part -- sign, exponent
 * and the top 10 fraction bits; the low 13 fraction bits are dropped (a
 * reading of the hardware, pinned by the tests). MN-major TF32 operands are
 * staged in the 128-byte swizzle with 32-byte atoms (GEMM_SWIZZLE_128B_ATOM32,
 * descriptor code 1): kind::tf32 reads an MN-major operand in that layout and
 * as zeros in SW128 (measured); K-major TF32 operands use the 32/64/128-byte
 * swizzles of the 16-bit types. */
gemm_status_t gemm_ex(int in_type, int64_t M, int64_t N, int64_t K,
                      const void *A, gemm_major_t a_major, int64_t lda,
                      const void *B, gemm_major_t b_major, int64_t ldb,
                      const void *C, int64_t ldc,
                      void *D, int64_t ldd, gemm_out_t d_type,
                      float alpha, float beta, const gemm_options_t *opts,
                      gemm_stream_t stream);

/* 8-bit float operand formats (tcgen05.mma kind::f8f6f4). */
typedef enum { GEMM_FP8_E4M3 = 0, GEMM_FP8_E5M2 = 1 } gemm_fp8_t;

/*
 * gemm_fp8 / gemm_fp8_ex: the same GEMM with 8-bit float operands, A and B
 * each E4M3 or E5M2 (they may differ), fp32 accumulation, output d_type.
 * The descriptors are the same as for 16-bit operands: one 16-byte core-matrix
 * cell holds 16 fp8 values ("LBO, SBO and SWZ for a tcgen05 tile", section 4)
 * and one MMA consumes 32 of them along K. Leading dimensions lda and ldb are
 * counted in elements (bytes) and must be multiples of 16; the other rules
 * are those above. opts may be NULL.
 */
gemm_status_t gemm_fp8(int64_t M, int64_t N, int64_t K,
                       const void *A, gemm_fp8_t a_format, gemm_major_t a_major, int64_t lda,
                       const void *B, gemm_fp8_t b_format, gemm_major_t b_major, int64_t ldb,
                       const void *C, int64_t ldc,
                       void *D, int64_t ldd, gemm_out_t d_type,
                       float alpha, float beta, gemm_stream_t stream);

gemm_status_t gemm_fp8_ex(int64_t M, int64_t N, int64_t K,
                          const void *A, gemm_fp8_t a_format, gemm_major_t a_major, int64_t lda,
                          const void *B, gemm_fp8_t b_format, gemm_major_t b_major, int64_t ldb,
                          const void *C, int64_t ldc,
                          void *D, int64_t ldd, gemm_out_t d_type,
                          float alpha, float beta, const gemm_options_t *opts,
                          gemm_stream_t stream);

/*
 * gemm_mxfp8: block-scaled fp8 GEMM (MXFP8: tcgen05 kind::mxf8f6f4 with
 * scale_vec::1X; "06 Blackwell Tensor Core - tcgen05 MMA", block-scaled
 * MMA: scale factors go from global memory to shared memory, then by
 * tcgen05.cp into TMEM, where the MMA reads them next to A and B).
 *   D = alpha * sum_k (sa[m, k/32] * A[m,k]) * (sb[n, k/32] * B[k,n]) + beta * C
 * A and B are E4M3 or E5M2 exactly as for gemm_fp8_ex; every 32 consecutive
 * elements of K of a row of A (column of B) share one scale, an 8-bit E8M0
 * code e meaning 2^(e - 127) (255 is NaN). The scales are stored in 512-byte
 * atoms, each covering 128 rows (of A; columns of B) x 4 scale blocks (128
 * elements of K): row r and K element k live in atom
 * (r / 128) * ceil(K / 128) + k / 128, at byte
 * 16 * (r % 32) + 4 * ((r % 128) / 32) + (k / 32) % 4 of it -- the layout
 * tcgen05.cp copies into TMEM, replicated over the four lane quarters.
 * SFA and SFB are device pointers, 16-byte aligned, of
 * gemm_mx_scale_bytes(M, K) and gemm_mx_scale_bytes(N, K) bytes; entries
 * for rows past M (N) or blocks past K are read and multiply only zeros, so
 * they must not be NaN (255).
 * Tiles: CTA pairs sharing a 256 x 256 tile (the default from M, N >= 2048;
 * one accumulator buffer, so each tile's epilogue is not overlapped and
 * stream_k is not applied), single CTAs of 128 x 128 (the default below
 * that), or pairs sharing 256 x 128 (cta_group 2 with tile_n 128). In a
 * pair each CTA holds the scales of its own A rows and a copy of all the
 * tile's B scales. 256
 * elements of K per pipeline stage (single CTAs may ask block_k = 128);
 * options asking for other tiles return GEMM_ERR_UNSUPPORTED. stream_k
 * applies as for gemm_ex.
 */
gemm_status_t gemm_mxfp8(int64_t M, int64_t N, int64_t K,
                         const void *A, gemm_fp8_t a_format, gemm_major_t a_major, int64_t lda,
                         const void *SFA,
                         const void *B, gemm_fp8_t b_format, gemm_major_t b_major, int64_t ldb,
                         const void *SFB,
                         const void *C, int64_t ldc,
                         void *D, int64_t ldd, gemm_out_t d_type,
                         float alpha, float beta, const gemm_options_t *opts,
                         gemm_stream_t stream);

/* Bytes of one scale tensor of gemm_mxfp8 for `rows` rows (M for SFA, N for
 * SFB) and K: ceil(rows / 128) * ceil(K / 128) * 512; 0 if either is <= 0. */
size_t gemm_mx_scale_bytes(int64_t rows, int64_t K);

/* Block-scaled fp4 formats of gemm_fp4 (E2M1 elements in both). */
typedef enum {
    GEMM_FP4_NVFP4 = 0, /* one UE4M3 scale per 16 elements of K (kind::mxf4nvf4, scale_vec::4X) */
    GEMM_FP4_MXFP4 = 1  /* one E8M0 scale per 32 elements of K (kind::mxf4, scale_vec::2X) */
} gemm_fp4_scale_t;

/*
 * gemm_fp4: block-scaled fp4 GEMM, the fp4 members of the block-scaled MMA
 * family of "06 Blackwell Tensor Core - tcgen05 MMA" (scales through
 * tcgen05.cp into TMEM, as for gemm_mxfp8).
 *   D = alpha * sum_k (sa[m, k/b] * A[m,k]) * (sb[n, k/b] * B[k,n]) + beta * C
 * with block b = 16 (NVFP4) or 32 (MXFP4). A (M x K) and B (stored N x K)
 * are K-major, E2M1 packed two to a byte: element 2i of a row in the low
 * nibble of byte i, 2i+1 in the high nibble. K, lda and ldb count elements;
 * K must be even and lda, ldb multiples of 32 (16-byte rows). Scale codes:
 * UE4M3 (unsigned E4M3: 2^(e-7) * (1 + m/8), e = 0 subnormal) for NVFP4,
 * E8M0 (2^(e-127)) for MXFP4, in the 512-byte atoms of gemm_mxfp8, one atom
 * per 128 rows x 4 blocks: row r and element k live in atom
 * (r / 128) * ceil(K / (4b)) + k / (4b), at byte
 * 16 * (r % 32) + 4 * ((r % 128) / 32) + (k / b) % 4. SFA and SFB hold
 * gemm_fp4_scale_bytes(M, K, kind) and gemm_fp4_scale_bytes(N, K, kind)
 * bytes, 16-byte aligned; entries for rows past M (N) or blocks past K
 * multiply only zeros but must be finite scales (a NaN code there, UE4M3
 * 0x7F or E8M0 255, makes the whole result NaN). Tiles: 256 x 256 CTA pairs
 * with one accumulator buffer (default from M, N >= 2048; cta_group 2) or
 * single CTAs of 128 x 128; stream_k (single CTAs)
 * applies as for gemm_ex; other tile options return GEMM_ERR_UNSUPPORTED.
 */
gemm_status_t gemm_fp4(int64_t M, int64_t N, int64_t K,
                       const void *A, int64_t lda, const void *SFA,
                       const void *B, int64_t ldb, const void *SFB,
                       gemm_fp4_scale_t kind,
                       const void *C, int64_t ldc,
                       void *D, int64_t ldd, gemm_out_t d_type,
                       float alpha, float beta, const gemm_options_t *opts,
                       gemm_stream_t stream);

/* Bytes of one scale tensor of gemm_fp4 for `rows` rows and K elements:
 * ceil(rows / 128) * ceil(K / (4 * block)) * 512; 0 for bad arguments. */
size_t gemm_fp4_scale_bytes(int64_t rows, int64_t K, gemm_fp4_scale_t kind);

/*
 * Grouped GEMM: num_problems independent problems in one launch. The
 * host list is read during the call; the library writes the device-side
 * problem list, one TMA descriptor per operand per problem and the tile
 * prefix sums into `workspace` (device memory owned by the caller, at
 * least gemm_grouped_workspace_size(num_problems) bytes, 128-byte
 * aligned) with an asynchronous copy on `stream`, then launches one
 * persistent kernel whose scheduler walks the concatenated tile list.
 * The workspace must stay untouched until the launch completes.
 */
size_t gemm_grouped_workspace_size(int num_problems);

gemm_status_t gemm_bf16_grouped(const gemm_problem_t *problems, int num_problems,
                                gemm_major_t a_major, gemm_major_t b_major,
                                gemm_out_t d_type, float alpha, float beta,
                                void *workspace, size_t workspace_bytes,
                                gemm_stream_t stream);

gemm_status_t gemm_f16_grouped(const gemm_problem_t *problems, int num_problems,
                               gemm_major_t a_major, gemm_major_t b_major,
                               gemm_out_t d_type, float alpha, float beta,
                               void *workspace, size_t workspace_bytes,
                               gemm_stream_t stream);

/* The grouped call with explicit options (opts may be NULL; tile_m, timeout
 * and flags as for gemm_ex). in_type: 0 fp16, 1 bf16. Without a cta_group
 * option, lists whose widest problem has N >= 2048 and whose tallest has
 * M >= 256 run on CTA pairs (256 x 256 tiles), others on single CTAs. */
gemm_status_t gemm_grouped_ex(int in_type, const gemm_problem_t *problems, int num_problems,
                              gemm_major_t a_major, gemm_major_t b_major,
                              gemm_out_t d_type, float alpha, float beta,
                              void *workspace, size_t workspace_bytes,
                              const gemm_options_t *opts, gemm_stream_t stream);

/*
 * gemm_bf16_grouped_noalloc: the grouped bf16 GEMM for callers that cannot
 * allocate device memory when they launch it: programs whose allocator has
 * reserved the whole device and forbids side allocations, plug-ins that a
 * host runtime hands only their input and output buffers, and real-time
 * loops that may not block in the driver's allocator (cudaMalloc can
 * synchronise the device). There is no counterpart on the pages; it is a
 * service of this library. Instead of a caller workspace, the problem table
 * and TMA descriptors go into a fixed array inside the library (about 68 KB,
 * room for GEMM_NOALLOC_MAX_PROBLEMS problems) that every GPU which loads the
 * library keeps until the process exits. The call allocates no device
 * memory and calls no allocating library routine; the table is staged in a
 * fixed host array and copied to the device array with cudaMemcpyAsync on
 * `stream` before the kernel launch.
 *   - Same arguments and results as gemm_bf16_grouped, minus the workspace.
 *   - num_problems > GEMM_NOALLOC_MAX_PROBLEMS returns GEMM_ERR_INVALID_ARG
 *     and enqueues nothing.
 *   - Set-up: the first call on a device looks up the array's device address
 *     there (cudaGetSymbolAddress, with that device current) and keeps it.
 *     Make that first call before any stream capture begins.
 *   - All calls share the array and each call rewrites the part it uses, so
 *     calls whose kernels may overlap on the GPU (other streams, or no
 *     ordering between them) race: order them on one stream or synchronise.
 */
#define GEMM_NOALLOC_MAX_PROBLEMS 128

gemm_status_t gemm_bf16_grouped_noalloc(const gemm_problem_t *problems, int num_problems,
                                        gemm_major_t a_major, gemm_major_t b_major,
                                        gemm_out_t d_type, float alpha, float beta,
                                        gemm_stream_t stream);

/* ---------------------------------------------------------------------
 * Expert layers: routing, 8-bit integer products, weighted sums. Element
 * types are gemm_out_t codes. The calls follow the rules above: device
 * pointers owned by the caller, no allocation, asynchronous on `stream`,
 * errors returned before anything is enqueued. Unless a rule below says
 * otherwise, pointers need only the alignment of their elements and leading
 * dimensions only the length of a row. Rows that are quantised or summed, and
 * the sizes of products, end 8192 short of 2^31 (GEMM_ERR_UNSUPPORTED past it).
 * The kernels are launched so that each
 * may start while the kernel before it on the stream ends (programmatic
 * dependent launch); they wait for it before they touch memory. The second of
 * gemm_route_plan's two kernels reads the ids before it waits for the first,
 * which lets it start only when what came before both has ended.
 * ------------------------------------------------------------------- */

typedef enum { GEMM_ROUTE_SOFTMAX = 0, GEMM_ROUTE_SIGMOID = 1 } gemm_score_t;

/*
 * How tokens choose experts (NULL: softmax scores, no groups, scale 1).
 *   score         scores s of a token from its logits l: softmax over the E
 *                 experts, or the sigmoid of each.
 *   groups        0 or 1: none. Otherwise the experts form this many groups
 *                 of E / groups neighbours (at most 32 groups; it divides E);
 *   group_top     a group's score is the sum of its group_top (1 or 2; 0
 *                 means 1) best s + bias;
 *   groups_kept   only the experts of the groups_kept best groups stay.
 *   renormalize   nonzero: a token's chosen scores are divided by their sum
 *                 (a sum of 0 leaves weights of 0).
 *   scale         factor on the weights; 0 means 1.
 */
typedef struct {
    int score;
    int groups;
    int group_top;
    int groups_kept;
    int renormalize;
    float scale;
} gemm_route_t;

#define GEMM_ROUTE_MAX_EXPERTS 1024
#define GEMM_ROUTE_MAX_K 32

/*
 * gemm_route: for each of T tokens, the k experts with the largest s + bias
 * (of the kept groups), best first, and their weights scale * s (/ the sum
 * of the chosen s). The bias (E fp32 values, or NULL) steers the choice and
 * is no part of the weights. Equal values go to the lower index; without a
 * bias the choice goes by the logits, whose order is that of the scores. The
 * scores that a choice with a bias (or between groups) compares and the
 * weights are good to fp32 rounding (a few units in the last place; a sigmoid
 * below 2^-126 counts as 0 in the weights).
 *   logits: T x E of l_type, row stride ldl. weights: T x k fp32; ids: T x k
 *   int32. 1 <= k <= min(E, GEMM_ROUTE_MAX_K), E <= GEMM_ROUTE_MAX_EXPERTS,
 *   k at most the experts of the kept groups.
 * A logit (or bias) of -inf or NaN is never chosen. Where fewer than k
 * experts are left (a padded token has none), the remaining ids are -1 and
 * their weights 0. A NaN logit, or under softmax one of +inf, makes all
 * weights of its token NaN; the ids stay valid (the choice takes a softmax
 * score of +inf as 1, that of the others beside it as 0).
 */
gemm_status_t gemm_route(int64_t T, int64_t E, const void *logits, gemm_out_t l_type, int64_t ldl,
                         const float *bias, int k, const gemm_route_t *route,
                         float *weights, int32_t *ids, gemm_stream_t stream);

/*
 * gemm_route_backward: the gradient of the logits from that of the weights,
 * for the ids that gemm_route chose (the choice itself, and with it the bias,
 * has none). dweights: T x k fp32; dlogits: T x E of l_type, row stride lddl,
 * written whole and not overlapping logits. Ids outside 0..E-1 carry nothing;
 * the others of a token are distinct. k and route as in the forward call (groups play no part).
 */
gemm_status_t gemm_route_backward(int64_t T, int64_t E, const void *logits, gemm_out_t l_type, int64_t ldl,
                                  int k, const gemm_route_t *route, const int32_t *ids,
                                  const float *dweights, void *dlogits, int64_t lddl, gemm_stream_t stream);

/*
 * gemm_route_plan: the order of the T * k (token, choice) pairs by expert,
 * for gemm_int8_grouped and the sums below. Pairs of one expert keep their
 * order (a stable counting sort: the result does not depend on timing).
 *   offsets  E + 1 int32: rows offsets[e] .. offsets[e+1]-1 are expert e's;
 *   slots    T x k int32: the row of each pair, -1 where its id is outside
 *            0..E-1;
 *   tokens   T * k int32: the token of each row, -1 past offsets[E].
 * T * k < 2^31. workspace: gemm_route_plan_workspace_size(T, E, k) bytes,
 * 4-byte aligned (may be NULL where that is 0); it needs no initialisation.
 */
size_t gemm_route_plan_workspace_size(int64_t T, int64_t E, int k);

gemm_status_t gemm_route_plan(int64_t T, int64_t E, int k, const int32_t *ids, int32_t *offsets,
                              int32_t *slots, int32_t *tokens, void *workspace, size_t workspace_bytes,
                              gemm_stream_t stream);

typedef enum { GEMM_QUANT_PLAIN = 0, GEMM_QUANT_GATED = 1 } gemm_quant_t;

/*
 * gemm_quantize_int8: rows to 8-bit integers, one scale a row:
 *   scales[m] = max_k |x[m,k]| / 127,  Q[m,k] = round(x[m,k] / scales[m])
 * in fp32, the scale as the product with the fp32 number nearest to 1/127 and
 * Q from the correctly rounded quotient (ties to even; a row of zeros has
 * scale 0). x[m,:] is row index[m] of X
 * (row m without an index), X having x_rows rows of x_type with stride ldx.
 * GEMM_QUANT_GATED: X rows are 2K wide, x = silu(X[:, :K]) * X[:, K:].
 * An index outside 0..x_rows-1 gives a row of zeros. A row that holds a
 * NaN or an infinity gets scale NaN and zeros, so that its products are NaN.
 * Q: M x K int8, row stride ldq (columns K..ldq-1 are not written).
 */
gemm_status_t gemm_quantize_int8(int64_t M, int64_t K, const void *X, gemm_out_t x_type, int64_t x_rows,
                                 int64_t ldx, const int32_t *index, gemm_quant_t mode,
                                 int8_t *Q, int64_t ldq, float *scales, gemm_stream_t stream);

/*
 * gemm_int8: D[m,n] = scale_a[m] * scale_b[n] * sum_k A[m,k] * B[n,k], the
 * product of 8-bit integers with a scale for each row (token) of A and each
 * row (channel) of B. A is M x K, B is N x K (both K-major), D is M x N of
 * d_type. sm_103a has no integer tcgen05 kind: the integers are widened to
 * fp16 on chip, where they and their products are exact, and summed in fp32,
 * exactly while partial sums stay below 2^24 in magnitude (any K <= 1024, and
 * far longer rows of quantised data), and to fp32 rounding beyond. Small
 * products of at most eight rows of A are summed in 32-bit integers instead,
 * which are exact for every K they are taken for (K < 2^17).
 * A and B 16-byte aligned, lda and ldb multiples of 16; K == 0 writes zeros.
 * Waits inside the tile kernels end after 2 s and 10 us for each 128 elements
 * of K that a CTA walks (GEMM_ERR_TIMEOUT by gemm_last_device_status).
 */
gemm_status_t gemm_int8(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, const float *scale_a,
                        const int8_t *B, int64_t ldb, const float *scale_b,
                        void *D, int64_t ldd, gemm_out_t d_type, gemm_stream_t stream);

/*
 * gemm_int8_grouped: the same over rows sorted by expert: rows offsets[e] ..
 * offsets[e+1]-1 of A (device memory, E + 1 int32, as gemm_route_plan writes
 * them, read by the kernel: no sizes pass through the host) multiply expert
 * e's matrix B + e * stride_b (N x K; stride_b in elements, a multiple of 16)
 * with its channel scales scale_b[e * N + n]. M is the room of A and D in
 * rows; rows from offsets[E] on are not written. Offsets that fall, or leave
 * 0..M, are clamped into it. 1 <= E <= GEMM_ROUTE_MAX_EXPERTS.
 */
gemm_status_t gemm_int8_grouped(int64_t M, int64_t N, int64_t K, int64_t E, const int32_t *offsets,
                                const int8_t *A, int64_t lda, const float *scale_a,
                                const int8_t *B, int64_t ldb, int64_t stride_b, const float *scale_b,
                                void *D, int64_t ldd, gemm_out_t d_type, gemm_stream_t stream);

/*
 * gemm_route_combine: D[t,:] = sum_j weights[t,j] * Y[slots[t,j],:], summed
 * in fp32 in the order of j. Y has y_rows rows of N values of y_type (stride
 * ldy), D is T x N of d_type. Slots outside 0..y_rows-1 add nothing, whatever
 * their weight. 1 <= k <= GEMM_ROUTE_MAX_K.
 */
gemm_status_t gemm_route_combine(int64_t T, int64_t N, int k, const void *Y, gemm_out_t y_type, int64_t y_rows,
                                 int64_t ldy, const int32_t *slots, const float *weights,
                                 void *D, gemm_out_t d_type, int64_t ldd, gemm_stream_t stream);

/*
 * gemm_route_combine_backward: dY[slots[t,j],:] = weights[t,j] * dD[t,:] and
 * dweights[t,j] = sum_n dD[t,n] * Y[slots[t,j],n] (0 where the slot is
 * outside 0..y_rows-1). dY: y_rows rows of y_type, stride lddy; rows that no
 * slot names are left as they are. The slots are distinct, as
 * gemm_route_plan makes them. dD is T x N of d_type.
 */
gemm_status_t gemm_route_combine_backward(int64_t T, int64_t N, int k, const void *dD, gemm_out_t d_type,
                                          int64_t lddd, const void *Y, gemm_out_t y_type, int64_t y_rows,
                                          int64_t ldy, const int32_t *slots, const float *weights,
                                          void *dY, int64_t lddy, float *dweights, gemm_stream_t stream);

/* ---------------------------------------------------------------------
 * The ends of a training step: rows of a token table, the loss of a linear head
 * over a large vocabulary, and the balance loss of the routers. The rules of the
 * expert-layer calls above hold (element types, alignment, errors, overlapping
 * launches), but for what is said here.
 * ------------------------------------------------------------------- */

/*
 * gemm_cross_entropy: softmax cross entropy of the logits l = X W^T, which are
 * never written to memory:
 *   lse[t] = log sum_v exp(l[t,v]),  losses[t] = lse[t] - l[t, targets[t]]
 * X is T x K, W is V x K, of in_type (0 fp16, 1 bf16; both row-major and
 * 16-byte aligned, ldx and ldw multiples of 8, as for gemm_ex). A token whose
 * target is outside 0..V-1 (padding, a prompt that is not trained on) has no
 * loss: losses[t] and lse[t] are 0, whatever its row of X holds. Logits are
 * summed in fp32, by tensor cores whose additions truncate in parts of 512
 * elements of K at most (256 for T <= 128, 128 for T <= 2) and by rounded additions
 * from part to part; sums of exponentials, lse and losses are fp32, the loss
 * without the rounding of lse. A logit of +inf makes lse +inf, one of NaN NaN.
 * workspace: gemm_cross_entropy_workspace_size(T, V) bytes, 16-byte aligned,
 * in no particular state. More tokens never ask for less.
 */
size_t gemm_cross_entropy_workspace_size(int64_t T, int64_t V);

gemm_status_t gemm_cross_entropy(int in_type, int64_t T, int64_t V, int64_t K, const void *X, int64_t ldx,
                                 const void *W, int64_t ldw, const int32_t *targets, float *losses, float *lse,
                                 void *workspace, size_t workspace_bytes, gemm_stream_t stream);

/*
 * gemm_cross_entropy_backward: gradients of sum_t dlosses[t] * losses[t] +
 * dlse[t] * lse[t] (dlse NULL: no gradient of lse; a penalty on the normaliser
 * has one) from the lse that the forward call wrote:
 *   dl[t,v] = exp(l[t,v] - lse[t]) * (dlosses[t] + dlse[t]) - [v = targets[t]] * dlosses[t]
 *   dX = dl W  (T x K of dx_type),   dW = dl^T X  (V x K of dw_type; accumulate
 *   nonzero: added to what dW holds, the sum rounded once)
 * dX or dW may be NULL, when only the other is wanted. Both are written whole,
 * 16-byte aligned with rows of a multiple of 16 bytes; they do not overlap the
 * inputs. Tokens without a loss carry nothing: their rows of dX are 0 (for a
 * finite W), and what their rows of X, dlosses and dlse hold has no part in dW.
 * dl is computed for a piece of the vocabulary at a time and rounded to the
 * inputs' type for the tensor cores, after a division by the largest
 * |dlosses| + |dlse| (found on the GPU: any scaling of the loss that leaves it
 * above 1e-30 gives the same gradients, times it); for one or two tokens of
 * K <= 4096 it is not rounded. The logits are summed as in the forward call, so that
 * exp(l - lse) of a certain word is 1; dX and dW in fp32 by the tensor cores, whose
 * additions truncate (every 16 terms, by up to 2^-23 of the sum so far).
 * T == 0 leaves dX and writes zeros to dW (nothing with accumulate).
 * workspace: 256-byte aligned, in no particular state. The call takes the widest
 * pieces that it has room for, of at most 2^27 / T columns (a piece's dl then has
 * 256 MB): gemm_cross_entropy_backward_workspace_size(T, V, K, columns) bytes for
 * pieces of `columns` columns (rounded up to a multiple of 256, the least; 0: the
 * widest), on the current device; 0 for bad arguments or without a device. More
 * tokens never ask for less, so that room for the most serves fewer. The
 * widths' order of sums differs, so gradients may differ in their last bits.
 */
size_t gemm_cross_entropy_backward_workspace_size(int64_t T, int64_t V, int64_t K, int64_t columns);

gemm_status_t gemm_cross_entropy_backward(int in_type, int64_t T, int64_t V, int64_t K, const void *X, int64_t ldx,
                                          const void *W, int64_t ldw, const int32_t *targets, const float *lse,
                                          const float *dlosses, const float *dlse, void *dX, gemm_out_t dx_type,
                                          int64_t lddx, void *dW, gemm_out_t dw_type, int64_t lddw, int accumulate,
                                          void *workspace, size_t workspace_bytes, gemm_stream_t stream);

/*
 * gemm_route_balance: counts per expert and the balance loss of a router, for
 * each of S sequences (tokens offsets[s] .. offsets[s+1]-1; offsets: S + 1 int32
 * in device memory that do not fall, those outside 0..T taken as its ends; NULL:
 * S is 1 and the sequence is all T tokens). Of the tokens of a sequence those
 * are live that have an id in 0..E-1 (padded tokens, as gemm_route leaves them,
 * have none); for its n live tokens
 *   counts[s,e] = number of ids that are e,      tokens[s] = n,
 *   means[s,e]  = mean of p[t,e],
 *   losses[s]   = E * sum_e counts[s,e] / (k n) * means[s,e]
 * with p the token's softmax over the E experts, or its sigmoid scores over their
 * sum (route->score; its other fields, and a bias, have no part; NULL: softmax).
 * A perfect balance has loss 1; a sequence without live tokens has zeros. Scores
 * are exponentials and reciprocals of the special-function unit: within 2^-21 of
 * themselves for logits of up to 10 (below the token's largest one with softmax),
 * 2^-22 + 1.25 |l| 2^-24 in all; sums are fp32.
 * ids: T x k int32 as gemm_route writes them; logits: T x E of l_type, row
 * stride ldl. counts and means: S x E; all fp32 or int32. E, k as for gemm_route.
 * workspace: gemm_route_balance_workspace_size(T, E, S) bytes, 16-byte aligned,
 * in no particular state (may be NULL where that is 0). More tokens or sequences
 * never ask for less, so that room for the most serves fewer. Sums have a fixed order.
 */
size_t gemm_route_balance_workspace_size(int64_t T, int64_t E, int64_t S);

gemm_status_t gemm_route_balance(int64_t T, int64_t E, const void *logits, gemm_out_t l_type, int64_t ldl, int k,
                                 const gemm_route_t *route, const int32_t *ids, int64_t S, const int32_t *offsets,
                                 int32_t *counts, int32_t *tokens, float *means, float *losses, void *workspace,
                                 size_t workspace_bytes, gemm_stream_t stream);

/*
 * gemm_route_balance_backward: the gradient of the logits from that of the
 * losses (S fp32 values), with the counts and tokens that the forward call wrote;
 * counts carry no gradient. dlogits: T x E of l_type, row stride lddl, not
 * overlapping logits. accumulate nonzero: added to what dlogits holds (such as
 * gemm_route_backward's gradient). Rows of tokens that are not live get zeros
 * (accumulate: stay as they are); rows of tokens in no sequence are not written.
 */
gemm_status_t gemm_route_balance_backward(int64_t T, int64_t E, const void *logits, gemm_out_t l_type, int64_t ldl,
                                          int k, const gemm_route_t *route, const int32_t *ids, int64_t S,
                                          const int32_t *offsets, const int32_t *counts, const int32_t *tokens,
                                          const float *dlosses, void *dlogits, int64_t lddl, int accumulate,
                                          gemm_stream_t stream);

/*
 * gemm_embed: D[t,:] = scale * table[ids[t],:], rows of N values; zeros where
 * the id is outside 0..V-1. table: V x N of t_type, row stride ldt; D: T x N of
 * d_type, row stride ldd; ids: T int32. The product is rounded once.
 */
gemm_status_t gemm_embed(int64_t T, int64_t N, int64_t V, const int32_t *ids, const void *table, gemm_out_t t_type,
                         int64_t ldt, float scale, void *D, gemm_out_t d_type, int64_t ldd, gemm_stream_t stream);

/*
 * gemm_embed_backward: dtable[v,:] = scale * sum of dD[t,:] over the tokens t
 * with ids[t] = v, in a fixed order, in fp32, rounded once. dtable is V x N of
 * t_type, written whole (rows that no id names get zeros); accumulate nonzero:
 * the sums are added to what it holds (a tied head's dW, say) and rows that no
 * id names are not touched. dD: T x N of d_type, row stride lddd. Ids outside
 * 0..V-1 carry nothing. scale is finite.
 * workspace: gemm_embed_backward_workspace_size(T, N, V) bytes, 256-byte
 * aligned, in no particular state (may be NULL where that is 0). More tokens
 * never ask for less, so that room for the most serves fewer.
 */
size_t gemm_embed_backward_workspace_size(int64_t T, int64_t N, int64_t V);

gemm_status_t gemm_embed_backward(int64_t T, int64_t N, int64_t V, const int32_t *ids, const void *dD,
                                  gemm_out_t d_type, int64_t lddd, float scale, void *dtable, gemm_out_t t_type,
                                  int64_t lddt, int accumulate, void *workspace, size_t workspace_bytes,
                                  gemm_stream_t stream);

/* Synchronises `stream`, reads the device status word of this library,
 * clears it, and returns GEMM_OK or GEMM_ERR_TIMEOUT (GEMM_ERR_CUDA if the
 * read fails). `detail` (may be NULL) receives the raw word: bits 0-7 the
 * role that gave up (1 producer, 2 MMA, 3 epilogue, 4 scale copier of the
 * block-scaled kinds, 5 launch setup: 10 in bits 8-15 means the dynamic
 * shared memory was not 1024-byte aligned, 6 a converter warp of the 8-bit
 * integer products), bits 8-15 the wait. */
gemm_status_t gemm_last_device_status(gemm_stream_t stream, uint32_t *detail);

const char *gemm_status_string(gemm_status_t status);

/* Number of this library's kernels launched since the library loaded. */
uint64_t gemm_launch_count(void);

/* ---------------------------------------------------------------------
 * Inspection entry points (tests): they expose the device-side builders
 * so their output can be compared bit for bit with an independent model.
 * ------------------------------------------------------------------- */

/*
 * Runs the device-side descriptor builder on the GPU and writes, for each
 * of the n_slices K=16 slices of one operand stage, the 64-bit shared-
 * memory matrix descriptor the GEMM kernel would hand to tcgen05.mma
 * ("LBO, SBO and SWZ for a tcgen05 tile", section 3: start, LBO, SBO, MBO
 * and SWZ fields), followed by the 32-bit instruction descriptor for
 * (M = 128 * cta_group, N = tile_n, in_type, f32 accumulate, majors) in the
 * low half of word n_slices. `out` is device memory of n_slices + 1 words.
 *   major: gemm_major_t of the operand; swizzle: gemm_swizzle_t (not AUTO);
 *   rows: MN extent of the stage (128 for A; tile_n or tile_n/2 for B);
 *   bk: K extent of the stage (32 or 64); stage_addr: shared-memory byte
 *   address of the stage (1024-aligned).
 */
gemm_status_t gemm_debug_descriptors(int major, int swizzle, int rows, int bk,
                                     uint32_t stage_addr, int n_slices,
                                     int cta_group, int tile_n, int in_type,
                                     int a_major, int b_major,
                                     uint64_t *out, gemm_stream_t stream);

/*
 * Loads one operand stage exactly as the GEMM producer does (TMA boxes in
 * the given swizzle into a 1024-aligned shared buffer) and copies the raw
 * shared-memory bytes to `out` (device memory, rows * bk * 2 bytes).
 *   src: device matrix of 16-bit elements, stored with leading dimension ld
 *   (K-major: rows_total x K with K contiguous; MN-major: K x rows_total
 *   with the MN index contiguous); (mn0, k0): the stage's origin.
 */
gemm_status_t gemm_debug_stage_image(const void *src, int major, int swizzle,
                                     int64_t rows_total, int64_t k_total, int64_t ld,
                                     int rows, int bk, int64_t mn0, int64_t k0,
                                     void *out, gemm_stream_t stream);

/*
 * Host-side tile plan (no GPU needed): the configuration a call would launch
 * on a device with `sms` SMs. kind: 0 fp16/bf16, 1 fp8, 2 MXFP8, 3 NVFP4,
 * 4 MXFP4 (K in elements), 5 TF32; grouped: nonzero for the grouped entry
 * points.
 * Writes 10 int32: cta_group, tile N, K per stage (bytes for fp4), rows per
 * CTA, swizzle bits of A and B (0 none, 1 32B, 2 64B, 3 128B, 4 128B with
 * 32-byte atoms), epilogue swizzle, group height, 1 when the tiles use
 * tcgen05.mma.ws, and 1 when two CTAs share B by multicast. Returns the
 * status the call's planning would.
 */
gemm_status_t gemm_debug_plan(int64_t M, int64_t N, int64_t K, int kind, int a_major, int b_major, int grouped,
                              const gemm_options_t *opts, int sms, int32_t *out);

/*
 * Host-side listing of the stream-K schedule (no GPU needed): the split the
 * library would choose for `tiles` tiles of `kb_per_tile` K blocks on a
 * grid of `clusters` clusters under stream_k `mode`, and the units of
 * cluster `cluster` in the order its roles run them -- the same code the
 * kernel's roles execute. Writes 6 int32 per unit to `out` (room for
 * max_units): tile, first K block, end K block (-1: the whole tile), kind
 * (0 whole, 1 contributor, 2 head), and for a head the first and last
 * contributing cluster (else 0, -1). Returns the number of units, or -1
 * when the launch would stay data-parallel (no units listed).
 */
int gemm_debug_streamk_units(int mode, int64_t tiles, int clusters, int kb_per_tile, int cluster,
                             int32_t *out, int max_units);

/*
 * Host-side plan of gemm_int8 (E = 0) and gemm_int8_grouped on a device with
 * `sms` SMs (no GPU needed). Writes 5 int32: kind (0 the integer kernel for few
 * tokens, 1 tiles with channels on the MMA's M side, 2 wide tiles), tokens and
 * channels of a tile, CTAs that share a tile's K, and the bound of a wait in
 * ms. Kind 0 has no tiles and no waits: M tokens, the others 0.
 */
gemm_status_t gemm_debug_int8_plan(int64_t M, int64_t N, int64_t K, int64_t E, int sms, int32_t *out);

/*
 * Host-side plan of gemm_cross_entropy_backward on a device with `sms` SMs (no GPU
 * needed) in a workspace of workspace_bytes. Writes 6 int64: the bytes that
 * gemm_cross_entropy_backward_workspace_size would return for pieces of `columns`,
 * those that the call would use of the workspace (more than it has: the call
 * refuses it), CTAs of a tile, pieces of the vocabulary, columns of a piece and
 * parts of dX. One or two tokens without tiles have 0 in the last four.
 */
gemm_status_t gemm_debug_cross_entropy_plan(int64_t T, int64_t V, int64_t K, int64_t columns, int sms,
                                            uint64_t workspace_bytes, int64_t *out);

/*
 * Host-side listing of the units of one launch of the cross entropy calls (no GPU
 * needed), by the code that deals them out and that the kernel's roles walk: of
 * the forward call (want 0) or of a backward call for dX (1), dW (2) or both (3)
 * in pieces of `columns` (0: the widest): `piece`'s gradients and the next piece's
 * dl (-1: dl alone). Writes 8 int32 for each unit (room for max_units): the
 * cluster, the product (0 dX, 1 dW, 2 logits), and the first and end of its
 * rows, columns and K, clipped to the product's. Returns the number of units, or
 * -1 for bad arguments and for tokens that have no tiles.
 */
int64_t gemm_debug_cross_entropy_units(int64_t T, int64_t V, int64_t K, int64_t columns, int sms, int64_t piece,
                                       int want, int32_t *out, int64_t max_units);

/* Test hook: the next GEMM launch makes its MMA warp wait on a barrier
 * that nothing arrives at, with a wait bound of `timeout_ms`; every role
 * then gives up and the kernel exits with GEMM_ERR_TIMEOUT recorded. */
void gemm_debug_inject_timeout(int timeout_ms);

/* The same for a chosen role: 1 the TMA producer (in both CTAs of a pair,
 * before it issues any load), 2 the MMA issuer; in the tiles of the 8-bit
 * integer products also 3 the epilogue of tiles that are not wide, and 6 the
 * converters (a launch that has no such role is not affected). Other roles
 * are ignored. The status word then names that role
 * with wait code 6 (injected), in the integer products' tiles that or a role
 * that waits for it. Where CTAs share a tile's K, role 3 instead leaves out the
 * others' sums, and the first CTA's epilogue gives up on them (wait code 13). */
void gemm_debug_inject_timeout_at(int timeout_ms, int role);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_GB300_H */
