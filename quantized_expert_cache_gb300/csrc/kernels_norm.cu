// Residual addition, root-mean-square norm and the int8 activation format in
// one pass over a token's row.
//
//   s = x + res (binary32), d_sum = s rounded to the stream's type
//   y = s * rsqrt(mean(s^2) + eps) * weight
//   per block of 32: d = binary16(amax|y| / 127), q = clamp(rint(y / d))
//
// The norm is taken of the binary32 sum, not of its rounded copy: the rounding
// to 16 bits is only what a 16-bit residual stream stores.
//
// Bound: HBM.  Every input is read once and every output written once; a row
// stays in registers between the sum of squares and its outputs (of widths above
// 8192 packs it is read twice).  Measured: 12288 x 2880 fp32 with codes 90.6 us =
// 0.98 of a copy's rate, 4096 x 2048 without 21.0 us = 0.94; 16-bit rows with codes
// 8192 x 4096 61.5 us = 0.89, 12288 x 2880 68.9 = 0.84; one row of 2048 2.1 us, 32
// rows of 2880 bf16 2.4 us (latency; one pack a thread, 4.1 us with four).
// 16-bit rows of 1025 to 2048 elements at more than 256 tokens hold eight packs of
// 8 a lane, which do not fit the 64 registers that blocks of 1024 threads leave:
// 242 to 256 bytes a thread spill, 12288 x 2048 bf16 60.2 us = 0.68 (and rows of
// 16385 to 65536 spill 306 to 332).  Widths that are no multiple of 4 take single
// elements: 8192 x 4097 fp32 0.86, bf16 0.72.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Pack {
    T v[N];
};

// The block's int8 codes of the VEC values each lane holds (32 / VEC lanes to
// a block) and its scale, the arithmetic of quantize_block_warp.
template <int VEC>
__device__ __forceinline__ void quantize_lane(const float *y, int8_t *q, float &dd) {
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < VEC; ++j) amax = __uint_as_float(max(__float_as_uint(amax), __float_as_uint(fabsf(y[j]))));
    unsigned m = __float_as_uint(amax);  // non-negative floats order like their bits
#pragma unroll
    for (int o = 16 / VEC; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    dd = __half2float(__float2half_rn(__uint_as_float(m) / 127.0f));
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        int c = 0;
        if (dd != 0.0f) c = (int)fminf(fmaxf(rintf(y[j] / dd), -127.0f), 127.0f);
        q[j] = (int8_t)c;
    }
}

// One row per warp (WARP_ROW, blockDim.x / 32 rows to a CTA) or per CTA.
// Lane-interleaved packs of VEC elements; ITEMS packs a thread in registers.
template <typename T, int VEC, int ITEMS, bool WARP_ROW>
__global__ void __launch_bounds__(1024) rms_norm_kernel(NormParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int step = WARP_ROW ? 32 : blockDim.x;
    const int first = WARP_ROW ? lane : threadIdx.x;
    const size_t row = WARP_ROW ? (size_t)blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
    if (WARP_ROW && row >= (size_t)p.n_tokens) return;
    const size_t base = row * (size_t)p.width;
    const T *x = (const T *)p.x + base, *res = p.res ? (const T *)p.res + base : nullptr;
    T *sum = p.sum ? (T *)p.sum + base : nullptr;
    const int nv = p.width / VEC;
    using PT = Pack<T, VEC>;
    using PF = Pack<float, VEC>;

    float s[ITEMS][VEC];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int v = first + i * step;
        PT a{}, b{};
        if (v < nv) {
            a = *((const PT *)x + v);
            if (res) b = *((const PT *)res + v);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[i][j] = to_f32<T>(a.v[j]) + to_f32<T>(b.v[j]);
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss = fmaf(s[i][j], s[i][j], ss);
    ss = warp_sum_f(ss);
    if (!WARP_ROW) {
        __shared__ float part[32];
        if (lane == 0) part[warp] = ss;
        __syncthreads();
        ss = warp_sum_f(lane < (int)(blockDim.x >> 5) ? part[lane] : 0.0f);
    }
    const float r = 1.0f / sqrtf(ss / (float)p.width + p.eps);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int v = first + i * step;
        const bool on = v < nv;
        PF g{};
        if (on) g = *((const PF *)p.weight + v);
        PF y;
#pragma unroll
        for (int j = 0; j < VEC; ++j) y.v[j] = s[i][j] * r * g.v[j];
        if (on && sum) {
            PT o;
#pragma unroll
            for (int j = 0; j < VEC; ++j) o.v[j] = from_f32<T>(s[i][j]);
            *((PT *)sum + v) = o;
        }
        if (on && p.y) *((PF *)(p.y + base) + v) = y;
        if (p.q) {
            // whole blocks only (width % 32 == 0): a block's lanes agree on `on`
            Pack<int8_t, VEC> q;
            float dd;
            quantize_lane<VEC>(y.v, q.v, dd);
            if (on) {
                *((Pack<int8_t, VEC> *)(p.q + base) + v) = q;
                if (lane % (32 / VEC) == 0) p.d[base / 32 + (size_t)v * VEC / 32] = __float2half_rn(dd);
            }
        }
    }
}

// Rows too wide for registers: one CTA a row, the inputs read twice.
template <typename T>
__global__ void __launch_bounds__(1024) rms_norm_wide_kernel(NormParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t base = (size_t)blockIdx.x * p.width;
    const T *x = (const T *)p.x + base, *res = p.res ? (const T *)p.res + base : nullptr;
    T *sum = p.sum ? (T *)p.sum + base : nullptr;
    float ss = 0.0f;
    // (unsigned: the step past the last element of the widest row needs the 32nd bit)
    const unsigned n = (unsigned)p.width;
    for (unsigned v = threadIdx.x; v < n; v += blockDim.x) {
        const float s = to_f32<T>(x[v]) + (res ? to_f32<T>(res[v]) : 0.0f);
        ss = fmaf(s, s, ss);
    }
    ss = warp_sum_f(ss);
    __shared__ float part[32];
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = warp_sum_f(lane < (int)(blockDim.x >> 5) ? part[lane] : 0.0f);
    const float r = 1.0f / sqrtf(ss / (float)p.width + p.eps);
    for (unsigned v0 = threadIdx.x - lane; v0 < n; v0 += blockDim.x) {
        const unsigned v = v0 + lane;
        const bool on = v < n;
        const float s = on ? to_f32<T>(x[v]) + (res ? to_f32<T>(res[v]) : 0.0f) : 0.0f;
        const float y = on ? s * r * p.weight[v] : 0.0f;
        if (on && sum) sum[v] = from_f32<T>(s);
        if (on && p.y) p.y[base + v] = y;
        if (p.q) {
            int8_t q;
            float dd;
            quantize_lane<1>(&y, &q, dd);
            if (on) {
                p.q[base + v] = q;
                if (lane == 0) p.d[(base + v) / 32] = __float2half_rn(dd);
            }
        }
    }
}

template <typename K>
int launch_pdl(K kernel, unsigned grid, unsigned block, const NormParams &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, kernel, p);
}

// (if constexpr: only the kernels that a call can reach are compiled)
template <typename T, int VEC>
int launch_typed(const NormParams &p, cudaStream_t st) {
    const int nv = p.width / VEC;
    const unsigned T_ = (unsigned)p.n_tokens;
    const bool few = p.n_tokens <= 256;
    // one warp a row: no barrier, and short rows share a CTA
    if (nv <= 32) return launch_pdl(rms_norm_kernel<T, VEC, 1, true>, (T_ + 7) / 8, 256, p, st);
    if (nv <= 64) return launch_pdl(rms_norm_kernel<T, VEC, 2, true>, (T_ + 7) / 8, 256, p, st);
    if (nv <= 128) return launch_pdl(rms_norm_kernel<T, VEC, 4, true>, (T_ + 7) / 8, 256, p, st);
    if (nv <= 256 && !few) return launch_pdl(rms_norm_kernel<T, VEC, 8, true>, (T_ + 7) / 8, 256, p, st);
    // one CTA a row
    auto threads = [&](int items) { return (unsigned)(((nv + items - 1) / items + 31) / 32 * 32); };
    if constexpr (VEC < 8)  // (packs of 8 are for many rows)
        if (nv <= 1024 && few) return launch_pdl(rms_norm_kernel<T, VEC, 1, false>, T_, threads(1), p, st);
    if constexpr (VEC == 1) {
        if (nv <= 512) return launch_pdl(rms_norm_kernel<T, VEC, 16, true>, (T_ + 7) / 8, 256, p, st);
    } else {
        if (nv <= 512) return launch_pdl(rms_norm_kernel<T, VEC, 2, false>, T_, threads(2), p, st);
    }
    if (nv <= 2048) return launch_pdl(rms_norm_kernel<T, VEC, 4, false>, T_, threads(4), p, st);
    if (nv <= 8192) return launch_pdl(rms_norm_kernel<T, VEC, 8, false>, T_, threads(8), p, st);
    return launch_pdl(rms_norm_wide_kernel<T>, T_, 1024, p, st);
}

template <typename T>
int launch_rows(const NormParams &p, cudaStream_t st) {
    const auto aligned = [](const void *q, size_t a) { return ((uintptr_t)q & (a - 1)) == 0; };
    if constexpr (sizeof(T) == 2)
        if (p.width % 8 == 0 && p.n_tokens > 256 && aligned(p.x, 16) && aligned(p.res, 16) && aligned(p.sum, 16) &&
            aligned(p.weight, 16) && aligned(p.y, 16) && aligned(p.q, 8))
            return launch_typed<T, 8>(p, st);
    const size_t e = 4 * sizeof(T);
    const bool vec = p.width % 4 == 0 && aligned(p.x, e) && aligned(p.res, e) && aligned(p.sum, e) &&
                     aligned(p.weight, 16) && aligned(p.y, 16) && aligned(p.q, 4);
    return vec ? launch_typed<T, 4>(p, st) : launch_typed<T, 1>(p, st);
}

}  // namespace

int launch_rms_norm(const NormParams &p, cudaStream_t st) {
    switch (p.dtype) {
        case 1: return launch_rows<__half>(p, st);
        case 2: return launch_rows<__nv_bfloat16>(p, st);
        default: return launch_rows<float>(p, st);
    }
}

}  // namespace moe
