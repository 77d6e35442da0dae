// Element access and reductions of the kernels that work on rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gemm_gb300.h"

namespace g300 {

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

// Calls fn with a value of the element type `type` names.
template <typename F>
inline gemm_status_t with_type(int type, F fn)
{
    switch (type) {
    case GEMM_OUT_F32: return fn(float());
    case GEMM_OUT_BF16: return fn(__nv_bfloat16());
    case GEMM_OUT_F16: return fn(__half());
    }
    return GEMM_ERR_INVALID_ARG;
}

}  // namespace g300
