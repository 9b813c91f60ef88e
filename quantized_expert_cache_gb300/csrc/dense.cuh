// Parts that the kernels of the 16-bit dense layers share: element types, the
// activations and their slopes, and what becomes of a finished sum.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace dense {

template <typename T>
__device__ __forceinline__ float value(T v);
template <>
__device__ __forceinline__ float value<float>(float v) { return v; }
template <>
__device__ __forceinline__ float value<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float value<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Element i of an array of a type known at run time.
__device__ __forceinline__ float load_as(const void *p, int dtype, size_t i) {
    if (dtype == 0) return ((const float *)p)[i];
    const unsigned short u = ((const unsigned short *)p)[i];
    return dtype == 1 ? __half2float(__ushort_as_half(u)) : __uint_as_float((unsigned)u << 16);
}
__device__ __forceinline__ void store_as(void *p, int dtype, size_t i, float v) {
    if (dtype == 0)
        ((float *)p)[i] = v;
    else
        ((unsigned short *)p)[i] =
            dtype == 1 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// act(z) and its slope: silu z s, s = 1 / (1 + exp(-z)); gelu z Phi(z), Phi the
// normal distribution's.  (Phi by erf: to 2^-24 or so of 1, not of itself.)
__device__ __forceinline__ float act_of(float z, int act) {
    if (act == kActSilu) return z / (1.0f + expf(-z));
    if (act == kActGelu) return 0.5f * z * (1.0f + erff(z * 0.70710678f));
    return z;
}
__device__ __forceinline__ float slope_of(float z, int act) {
    if (act == kActSilu) {
        const float s = 1.0f / (1.0f + expf(-z));
        return s * (1.0f + z * (1.0f - s));
    }
    if (act == kActGelu)
        return 0.5f * (1.0f + erff(z * 0.70710678f)) + z * 0.39894228f * expf(-0.5f * z * z);
    return 1.0f;
}

// A finished sum v of output row m (contiguous) and column n.
__device__ __forceinline__ void finish(const DenseOut &o, size_t m, size_t n, float bias, float v) {
    const size_t i = n * (size_t)o.ld + m;
    v += bias;
    if (o.pre) store_as(o.pre, o.dtype, i, v);
    v = act_of(v, o.act);
    if (o.res) v += load_as(o.res, o.dtype, i);
    store_as(o.out, o.dtype, i, v);
}

}  // namespace dense
}  // namespace moe
