// Host services of gemm_api.cu shared with the other entry-point units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

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

// Takes a pending timeout injection (gemm_debug_inject_timeout): the role
// that shall wait and its bound in ms, or 0.
int host_take_injection(int *timeout_ms);

// Counts `n` launched kernels in gemm_launch_count().
void host_count_launches(int n);

// A launch's status after it was enqueued, counted when it was.
inline gemm_status_t host_launched(int n = 1)
{
    if (cudaGetLastError() != cudaSuccess)
        return GEMM_ERR_CUDA;
    host_count_launches(n);
    return GEMM_OK;
}

inline int type_bytes(int type) { return type == GEMM_OUT_F32 ? 4 : 2; }

inline bool valid_type(int type) { return type == GEMM_OUT_F32 || type == GEMM_OUT_BF16 || type == GEMM_OUT_F16; }

inline bool aligned_to(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

constexpr int64_t kSizeLimit = (static_cast<int64_t>(1) << 31) - 1;

inline bool valid_size(int64_t n) { return n >= 0 && n <= kSizeLimit; }

// Strides below 2^40 bytes: row * stride stays within 64 bits.
inline bool valid_stride(int64_t ld, int esize) { return ld >= 0 && ld < (static_cast<int64_t>(1) << 40) / esize; }

}  // namespace g300
