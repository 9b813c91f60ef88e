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
// normal distribution's.  (Phi by erf: to 2^-24 or so of 1, not of itself; exp by the
// special-function unit: (4 + 2.4 |z|) 2^-24 of itself, its quotient 4 2^-24 more; s below
// 2^-126 is 0.)
__device__ __forceinline__ float act_of(float z, int act) {
    if (act == kActSilu) return __fdividef(z, 1.0f + __expf(-z));
    if (act == kActGelu) return 0.5f * z * (1.0f + erff(z * 0.70710678f));
    return z;
}
__device__ __forceinline__ float slope_of(float z, int act) {
    if (act == kActSilu) {
        const float s = __fdividef(1.0f, 1.0f + __expf(-z));
        return s * (1.0f + z * (1.0f - s));
    }
    if (act == kActGelu)
        return 0.5f * (1.0f + erff(z * 0.70710678f)) + z * 0.39894228f * __expf(-0.5f * z * z);
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

// The blocks' sums of a column, in a fixed order: the same bits every time.  A warp takes
// 8 columns at a time, every fourth block in a lane; `first` of `step` warps.
__device__ __forceinline__ void finish_sums(const float *parts, float *sums, int blocks, int cols, int first, int step,
                                            int lane) {
    for (long long c0 = 8ll * first; c0 < cols; c0 += 8ll * step) {
        const long long c = c0 + (lane & 7);
        float s = 0.0f;
        if (c < cols)
#pragma unroll 8
            for (int b = lane >> 3; b < blocks; b += 4) s += parts[(size_t)b * cols + c];
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        if (lane < 8 && c < cols) sums[c] = s;
    }
}

// Four elements from i, at once if the array allows it.
__device__ __forceinline__ void load4_as(const void *p, int dtype, size_t i, float *v) {
    if (dtype == 0) {
        const float4 f = *(const float4 *)((const float *)p + i);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
        const ushort4 u = *(const ushort4 *)((const unsigned short *)p + i);
        const unsigned short h[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = dtype == 1 ? __half2float(__ushort_as_half(h[j])) : __uint_as_float((unsigned)h[j] << 16);
    }
}
__device__ __forceinline__ void store4_as(void *p, int dtype, size_t i, const float *v) {
    if (dtype == 0) {
        *(float4 *)((float *)p + i) = float4{v[0], v[1], v[2], v[3]};
    } else {
        unsigned short h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h[j] = dtype == 1 ? __half_as_ushort(__float2half_rn(v[j])) : __bfloat16_as_ushort(__float2bfloat16_rn(v[j]));
        *(ushort4 *)((unsigned short *)p + i) = ushort4{h[0], h[1], h[2], h[3]};
    }
}

// Two values rounded to binary16 or bfloat16, the first in the low half.
__device__ __forceinline__ unsigned pair16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *(const unsigned *)&h;
}
__device__ __forceinline__ unsigned pairb16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *(const unsigned *)&h;
}

// The epilogue of four neighbours m of the result in a lane.
struct Epilogue {
    DenseOut o;    // (a copy: stores through its pointers could alias the original)
    int m, left;   // the lane's first row, rows from it to the end
    bool wide;     // the lane's four at once
    bool plain;    // sums as they are, all lanes' rows at once
    __device__ __forceinline__ Epilogue(const DenseOut &out, int M, int m_, size_t offset) : o(out), m(m_), left(M - m_) {
        if (offset) o.out = (float *)o.out + offset;  // (a K share's sums)
        const uintptr_t at = (uintptr_t)o.out | (uintptr_t)o.res | (uintptr_t)o.pre;
        wide = left >= 4 && o.ld % 4 == 0 && (at & (o.dtype == 0 ? 15 : 7)) == 0;
        plain = !o.pre && !o.res && o.act == kActNone && M == o.ld && M % (o.dtype == 0 ? 4 : 8) == 0 &&
                ((uintptr_t)o.out & 15) == 0;
    }
    // column n's finished sums, the bias among them
    __device__ __forceinline__ void column(const float *sums, int n) const {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = sums[j];
        const size_t i = (size_t)n * (size_t)o.ld + m;
        if (wide) {
            if (o.pre) store4_as(o.pre, o.dtype, i, v);
            if (o.act != kActNone)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = act_of(v[j], o.act);
            if (o.res) {
                float r[4];
                load4_as(o.res, o.dtype, i, r);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] += r[j];
            }
            store4_as(o.out, o.dtype, i, v);
        } else {
            // (every fourth element of a column a store: 4096 x 32003 x 2048 486 us, 32000 298)
#pragma unroll 1
            for (int j = 0; j < 4 && j < left; ++j) {
                float z = j == 0 ? v[0] : j == 1 ? v[1] : j == 2 ? v[2] : v[3];
                if (o.pre) store_as(o.pre, o.dtype, i + j, z);
                z = act_of(z, o.act);
                if (o.res) z += load_as(o.res, o.dtype, i + j);
                store_as(o.out, o.dtype, i + j, z);
            }
        }
    }
    // A warp's 32 rows (8 lanes, from 4 (lane & 7) on) of `cols` columns from n of N:
    // sums[column][32] in shared memory, four columns at a time.
    __device__ __forceinline__ void store(const float *sums, int cols, int n, int N, int lane) const {
        const int most = min(cols, N - n);
        if (plain && o.dtype != 0) {
            // rounded sums alone: eight neighbours a lane, eight columns at a time
            const int at = (lane & 3) * 8, m8 = m - (lane & 7) * 4 + at;
            if (left + m <= m8) return;
            unsigned short *out = (unsigned short *)o.out + (size_t)n * (size_t)o.ld + m8;
#pragma unroll 2
            for (int c = lane >> 2; c < most; c += 8) {
                const float4 f = *(const float4 *)(sums + c * 32 + at), g = *(const float4 *)(sums + c * 32 + at + 4);
                const uint4 u = o.dtype == 1 ? uint4{pair16(f.x, f.y), pair16(f.z, f.w), pair16(g.x, g.y), pair16(g.z, g.w)}
                                             : uint4{pairb16(f.x, f.y), pairb16(f.z, f.w), pairb16(g.x, g.y), pairb16(g.z, g.w)};
                *(uint4 *)(out + (size_t)c * o.ld) = u;
            }
            return;
        }
        if (left <= 0) return;
        if (plain) {
            float *out = (float *)o.out + (size_t)n * (size_t)o.ld + m;
#pragma unroll 2
            for (int c = lane >> 3; c < most; c += 4)
                *(float4 *)(out + (size_t)c * o.ld) = *(const float4 *)(sums + c * 32 + (lane & 7) * 4);
            return;
        }
#pragma unroll 1
        for (int c = lane >> 3; c < most; c += 4) {
            const float4 f = *(const float4 *)(sums + c * 32 + (lane & 7) * 4);
            const float v[4] = {f.x, f.y, f.z, f.w};
            column(v, n + c);
        }
    }
};

}  // namespace dense
}  // namespace moe
