// Host services of gemm_api.cu shared with the other entry-point units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/gemm_gb300.h"

namespace g300 {

// Current device, the device address of the library's status word, and the
// number of SMs.
gemm_status_t host_device(int *dev, unsigned int **status, int *sms);

// A tiled tensor map of rank 2 or 3: dims and box innermost first, strides (in
// bytes) of the outer dimensions, zero fill outside.
gemm_status_t host_encode_tiled(CUtensorMap *map, CUtensorMapDataType dt, int rank, const void *ptr,
                                const uint64_t *dims, const uint64_t *strides, const uint32_t *box,
                                CUtensorMapSwizzle swz);

// Role code of the converters of the 8-bit integer products in the status word,
// beside those of gemm_kernel.cuh.
constexpr unsigned int kRoleConvert = 6;

// Takes a pending timeout injection (gemm_debug_inject_timeout): the role
// that shall wait and its bound in ms, or 0.
int host_take_injection(int *timeout_ms);

// Counts `n` launched kernels in gemm_launch_count().
void host_count_launches(int n);

// Opt a kernel into its dynamic shared memory once per device (the attribute
// is per device; setting it on every launch costs host time on short GEMMs).
// `done` is the caller's per-variant record: one bit per device 0..127.
template <typename Kern>
cudaError_t ensure_smem_attribute(Kern kern, int bytes, std::atomic<uint64_t> (&done)[2])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 128)
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (done[dev >> 6].load(std::memory_order_acquire) & bit)
        return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        done[dev >> 6].fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

// Launches a kernel that may start while the kernel before it on the stream is
// still running (programmatic dependent launch). Such a kernel calls
// grid_start() before it touches memory that another kernel writes or reads:
// only its launch and what it sets up on chip overlap. (One reads earlier:
// plan_scatter_kernel its ids. The kernel before it, plan_count_kernel, lets it
// start after its own wait, so that what wrote the ids has ended.) With
// `cluster` > 0 it is launched in clusters of that many CTAs.
template <typename... Params, typename... Args>
inline gemm_status_t host_launch(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                                 unsigned cluster, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...) != cudaSuccess) {
        (void)cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    host_count_launches(1);
    return GEMM_OK;
}

#ifdef __CUDACC__
// The next kernel on the stream may be launched from here on (it waits in its
// own grid_start); the kernels before this one have finished on return, and
// their writes are visible. They were not when this kernel started, so it reads
// what others write with ordinary loads only: no __ldg, no __restrict__ inputs.
__device__ __forceinline__ void grid_start()
{
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
}
#endif

inline int type_bytes(int type) { return type == GEMM_OUT_F32 ? 4 : 2; }

inline bool valid_type(int type) { return type == GEMM_OUT_F32 || type == GEMM_OUT_BF16 || type == GEMM_OUT_F16; }

inline bool aligned_to(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

constexpr int64_t kSizeLimit = (static_cast<int64_t>(1) << 31) - 1;

inline bool valid_size(int64_t n) { return n >= 0 && n <= kSizeLimit; }

// Lengths that a kernel walks with 32-bit counters, whose steps (at most 4096
// columns) may pass the end once.
inline bool countable(int64_t n) { return n <= kSizeLimit - 8192; }

// Strides below 2^40 bytes, as tensor maps want them. That the rows which a
// call names exist, and so lie within 64 bits, is the caller's part.
inline bool valid_stride(int64_t ld, int esize) { return ld >= 0 && ld < (static_cast<int64_t>(1) << 40) / esize; }

}  // namespace g300
