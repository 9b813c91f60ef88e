// 16-bit dense layers: products of few tokens, and the preparation of operands for
// the tensor cores (kernels_dense_gemm.cu).
//
// Few tokens.  y = act(x W^T + bias) + res is bound by the read of W: a warp takes
// one or two rows of W (four warps a row where rows are few) and all tokens, its lanes
// neighbouring packs of 8 columns; products and sums in fp32.  Measured: one token on 512
// x 2048 1.9 us (latency), 512 x 8192 3.7 (8.7 with a warp a row), 65536 x 2048 40.9 = 0.96
// of a copy.
//
// Parts.  An fp32 operand (or one with a slope) goes to the tensor cores as 16-bit
// numbers, each the rounding of what the ones before leave; products of parts are further
// steps of the same sum.
//   fp32 results: three bfloat16 parts, all 24 bits (what lies below 2^-133 is lost), and
//     the products to 2^-24: 3 with a 16-bit operand, 6 of two fp32 ones.  (Two parts
//     and three products leave 3e-6 to 4.5e-6 of a gradient's norm, a plain fp32 product
//     about 1e-6.)  A gradient through a slope in binary16: two binary16 parts of its half (a
//     slope of 1.13 takes it past binary16's range), the second held 2^12 larger (22 bits,
//     or 2^-36).
//   16-bit results: two parts.
// A gradient that is 16-bit itself, without a slope, goes as it is.  Measured (the
// profiler's clock, cold): 4096 x 2048 fp32 in three parts 16 us for 84 MB; 1000 x 2880 fp16
// with gelu's slope in two 12 us for 23 MB: a warp has two tokens there, the second one's
// loads wait for the first one's slopes.
#include <algorithm>
#include <type_traits>

#include "dense.cuh"

namespace moe {
namespace {

using namespace dense;

template <typename T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Pack {
    T v[N];
};

// ---- few tokens ---------------------------------------------------------------
// ROWS rows of W and T tokens to KW warps (of a row's packs every KW-th 32), DEPTH
// packs of 8 columns in flight a row.
template <typename TX, typename TW, int T, int ROWS, int KW>
__global__ void __launch_bounds__(256) dense_few_kernel(DenseFew p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int DEPTH = 8 / ROWS, STEP = 32 * KW;
    static_assert(KW == 1 || ROWS == 1, "one row to several warps");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, packs = p.cols / 8;
    const size_t r0 = ((size_t)blockIdx.x * (8 / KW) + warp / KW) * ROWS;
    if (KW == 1 && r0 >= (size_t)p.rows) return;
    const TX *x = (const TX *)p.x;
    const TW *w[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)  // (rows past the end are the last one)
        w[r] = (const TW *)p.w + min(r0 + r, (size_t)p.rows - 1) * p.cols;
    float acc[ROWS][T];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[r][t] = 0.0f;
    for (int c0 = lane + 32 * (warp % KW); c0 < packs; c0 += STEP * DEPTH) {
        Pack<TW, 8> v[DEPTH][ROWS];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                v[d][r] = Pack<TW, 8>{};
                if (c0 + STEP * d < packs) *(uint4 *)&v[d][r] = __ldcs((const uint4 *)w[r] + c0 + STEP * d);
            }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (c0 + STEP * d >= packs) break;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const Pack<TX, 8> a = *((const Pack<TX, 8> *)(x + (size_t)t * p.cols) + c0 + STEP * d);
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int r = 0; r < ROWS; ++r)
                        acc[r][t] = fmaf(value<TX>(a.v[j]), value<TW>(v[d][r].v[j]), acc[r][t]);
            }
        }
    }
    float mine = 0.0f;  // lane i: row i / T, token i % T
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const float s = warp_sum_f(acc[r][t]);
            if (lane == r * T + t) mine = s;
        }
    if (KW > 1) {
        __shared__ float part[8][T];
        if (lane < T) part[warp][lane] = mine;
        __syncthreads();
        if (warp % KW != 0) return;
        if (lane < T)
#pragma unroll
            for (int k = 1; k < KW; ++k) mine += part[warp + k][lane];
    }
    if (lane < ROWS * T) {
        const size_t m = r0 + lane / T;
        if (m < (size_t)p.rows) finish(p.o, m, lane % T, p.o.bias ? p.o.bias[m] : 0.0f, mine);
    }
}

// ---- parts and column sums ------------------------------------------------------
// A CTA takes 256 columns (8 a lane) of some tokens, a warp every eighth of them.
// WIDE: rows of 16-byte packs; else neighbouring lanes take neighbouring columns.
constexpr int kSplitCols = 256;

template <typename T, typename P, int PARTS, bool WIDE>
__global__ void __launch_bounds__(256) dense_split_kernel(DenseSplit p, int block_tokens) {
    // (beside another kernel of the call, which started after all work before the call was
    // done and whose end is waited for below: this one's end then stands for both)
    if (!p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ float part_sum[8][kSplitCols];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int strips = (p.cols + kSplitCols - 1) / kSplitCols, strip = blockIdx.x % strips;
    const int block = blockIdx.x / strips;
    const int c0 = strip * kSplitCols;
    const auto col = [&](int j) { return c0 + (WIDE ? lane * 8 + j : j * 32 + lane); };
    const size_t t0 = (size_t)block * block_tokens, t1 = min(t0 + block_tokens, (size_t)p.n_tokens);
    float sum[8] = {};
    // a token's 8 columns of a lane, the next one's loads in flight
    struct Eight {
        Pack<T, 8> src, pre;
    };
    const auto load = [&](size_t t) {
        Eight e{};
        const T *src = (const T *)p.src + t * p.cols, *pre = (const T *)p.pre + t * p.cols;
        if (WIDE) {
            if (col(0) < p.cols) {
                e.src = *(const Pack<T, 8> *)(src + col(0));
                if (p.pre) e.pre = *(const Pack<T, 8> *)(pre + col(0));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (col(j) < p.cols) e.src.v[j] = src[col(j)];
                if (p.pre && col(j) < p.cols) e.pre.v[j] = pre[col(j)];
            }
        }
        return e;
    };
    Eight next{};
    if (t0 + warp < t1) next = load(t0 + warp);
    for (size_t t = t0 + warp; t < t1; t += 8) {
        float v[8], z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = value<T>(next.src.v[j]), z[j] = value<T>(next.pre.v[j]);
        if (t + 8 < t1) next = load(t + 8);
        if (p.pre)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], slope_of(z[j], p.act));  // (not fused into the sum)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += v[j];
        if (PARTS) {
            if constexpr (std::is_same<P, __half>::value) {
                if (p.pre)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] *= kDenseHold;
            }
            unsigned cut = 0;
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
                Pack<P, 8> o;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    o.v[j] = rounded<P>(v[j]);
                    if constexpr (std::is_same<P, __nv_bfloat16>::value) {
                        // values that round past bfloat16's range are cut, all their parts: no
                        // sum of the first ones is larger than the value
                        if (q == 0) cut |= isinf(value<P>(o.v[j])) && !isinf(v[j]) ? 1u << j : 0;
                        if (cut >> j & 1) o.v[j] = __ushort_as_bfloat16((unsigned short)(__float_as_uint(v[j]) >> 16));
                    }
                    const float left = v[j] - value<P>(o.v[j]);
                    // infinities and NaN are their first part
                    v[j] = isfinite(value<P>(o.v[j])) ? left : 0.0f;
                    if constexpr (std::is_same<P, __half>::value)
                        v[j] = fminf(fmaxf(v[j] * kDenseLowScale, -kDenseMost16), kDenseMost16);
                }
                P *dst = (P *)p.parts + (p.by_row ? t * PARTS + q : (size_t)q * p.n_tokens + t) * p.ld;
                if (WIDE) {
                    if (col(0) < p.cols) *(Pack<P, 8> *)(dst + col(0)) = o;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (col(j) < p.cols) dst[col(j)] = o.v[j];
                }
            }
        }
    }
    if (p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!p.sums) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) part_sum[warp][col(j) - c0] = sum[j];
    __syncthreads();
    const int c = c0 + threadIdx.x;
    if (c < p.cols) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += part_sum[w][threadIdx.x];
        p.ws_sums[(size_t)block * p.cols + c] = s;
    }
}

// Column sums alone, of what has no slope: the split's order of summation (and bits) with
// four tokens' loads of a warp in flight and no more registers than that.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) dense_columns_kernel(DenseSplit p, int block_tokens) {
    if (!p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ float part_sum[8][kSplitCols];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int strips = (p.cols + kSplitCols - 1) / kSplitCols, c0 = blockIdx.x % strips * kSplitCols;
    const int block = blockIdx.x / strips;
    const auto col = [&](int j) { return c0 + (WIDE ? lane * 8 + j : j * 32 + lane); };
    const size_t t0 = (size_t)block * block_tokens, t1 = min(t0 + block_tokens, (size_t)p.n_tokens);
    float sum[8] = {};
    for (size_t t = t0 + warp; t < t1; t += 32) {
        Pack<T, 8> v[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            v[d] = Pack<T, 8>{};
            const T *src = (const T *)p.src + (t + 8 * d) * p.cols;
            if (t + 8 * d >= t1) continue;
            if (WIDE) {
                if (col(0) < p.cols) v[d] = *(const Pack<T, 8> *)(src + col(0));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col(j) < p.cols) v[d].v[j] = src[col(j)];
            }
        }
#pragma unroll
        for (int d = 0; d < 4; ++d)
            if (t + 8 * d < t1)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += value<T>(v[d].v[j]);
    }
    if (p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
    for (int j = 0; j < 8; ++j) part_sum[warp][col(j) - c0] = sum[j];
    __syncthreads();
    const int c = c0 + threadIdx.x;
    if (c < p.cols) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += part_sum[w][threadIdx.x];
        p.ws_sums[(size_t)block * p.cols + c] = s;
    }
}

__global__ void __launch_bounds__(32) dense_sums_kernel(const float *part, float *sums, int blocks, int cols) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    finish_sums(part, sums, blocks, cols, blockIdx.x, gridDim.x, threadIdx.x);
}

// ---- K shares of a product -------------------------------------------------------
template <int VEC>
__global__ void __launch_bounds__(256) dense_join_kernel(const float *parts, int shares, size_t n, void *out, int dtype) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * VEC; i < n; i += (size_t)gridDim.x * 256 * VEC) {
        float v[VEC] = {};
#pragma unroll 4
        for (int s = 0; s < shares; ++s) {
            const Pack<float, VEC> p = *(const Pack<float, VEC> *)(parts + s * n + i);
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] += p.v[j];
        }
        if (VEC == 4)
            store4_as(out, dtype, i, v);
        else
            store_as(out, dtype, i, v[0]);
    }
}

template <typename K, typename... A>
int launch(K kernel, size_t grid, int threads, cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, typename P, int PARTS>
int launch_split(const DenseSplit &p, cudaStream_t st) {
    const int bt = dense_block_tokens(p.n_tokens), strips = (p.cols + kSplitCols - 1) / kSplitCols;
    const size_t grid = (size_t)strips * ((p.n_tokens + bt - 1) / bt);
    const bool wide = p.cols % 8 == 0 && (((uintptr_t)p.src | (uintptr_t)p.pre | (uintptr_t)p.parts) & 15) == 0;
    int rc;
    if (PARTS == 0 && !p.pre)
        rc = wide ? launch(dense_columns_kernel<T, true>, grid, 256, st, p, bt)
                  : launch(dense_columns_kernel<T, false>, grid, 256, st, p, bt);
    else
        rc = wide ? launch(dense_split_kernel<T, P, PARTS, true>, grid, 256, st, p, bt)
                  : launch(dense_split_kernel<T, P, PARTS, false>, grid, 256, st, p, bt);
    if (rc || !p.sums || !p.finish) return rc;
    return launch(dense_sums_kernel, (p.cols + 7) / 8, 32, st, (const float *)p.ws_sums, p.sums,
                  dense_sum_blocks(p.n_tokens), p.cols);
}

template <typename TX, typename TW, int ROWS, int KW>
int launch_few_rows(const DenseFew &p, cudaStream_t st) {
    const int rows = 8 / KW * ROWS;
    const size_t grid = ((size_t)p.rows + rows - 1) / rows;
    switch (p.n_tokens) {
        case 1: return launch(dense_few_kernel<TX, TW, 1, ROWS, KW>, grid, 256, st, p);
        case 2: return launch(dense_few_kernel<TX, TW, 2, ROWS, KW>, grid, 256, st, p);
        case 3: return launch(dense_few_kernel<TX, TW, 3, ROWS, KW>, grid, 256, st, p);
        default: return launch(dense_few_kernel<TX, TW, 4, ROWS, KW>, grid, 256, st, p);
    }
}

template <typename TX, typename TW>
int launch_few(const DenseFew &p, int n_sm, cudaStream_t st) {
    // four warps a row where rows are few and long, a warp a row while that leaves warps to
    // spare: more of them, shorter
    if (p.rows <= n_sm * 8 && p.cols >= 1024) return launch_few_rows<TX, TW, 1, 4>(p, st);
    return p.rows <= n_sm * 32 ? launch_few_rows<TX, TW, 1, 1>(p, st) : launch_few_rows<TX, TW, 2, 1>(p, st);
}

}  // namespace

// (1 part of a 16-bit type: a copy with aligned rows; 0: sums alone)
int launch_dense_split(const DenseSplit &p, cudaStream_t st) {
    using bf = __nv_bfloat16;
    switch (p.dtype * 4 + p.n_parts) {
        case 0: return launch_split<float, bf, 0>(p, st);
        case 2: return launch_split<float, bf, 2>(p, st);
        case 3: return launch_split<float, bf, 3>(p, st);
        case 4: return launch_split<__half, __half, 0>(p, st);
        case 5: return launch_split<__half, __half, 1>(p, st);
        case 6: return launch_split<__half, __half, 2>(p, st);
        case 8: return launch_split<bf, bf, 0>(p, st);
        case 9: return launch_split<bf, bf, 1>(p, st);
        case 10: return launch_split<bf, bf, 2>(p, st);
        case 11: return launch_split<bf, bf, 3>(p, st);
        default: return (int)cudaErrorInvalidValue;
    }
}

int launch_dense_join(const float *parts, int shares, size_t n, void *out, int dtype, int n_sm, cudaStream_t st) {
    const bool wide = n % 4 == 0 && ((uintptr_t)out & (dtype == 0 ? 15 : 7)) == 0;
    const size_t blocks = (n / (wide ? 4 : 1) + 255) / 256;
    const unsigned grid = (unsigned)std::max<size_t>(1, std::min<size_t>(blocks, (size_t)n_sm * 8));
    return wide ? launch(dense_join_kernel<4>, grid, 256, st, parts, shares, n, out, dtype)
                : launch(dense_join_kernel<1>, grid, 256, st, parts, shares, n, out, dtype);
}

int launch_dense_few(const DenseFew &p, int n_sm, cudaStream_t st) {
    if (p.w_dtype == 1) return launch_few<__half, __half>(p, n_sm, st);
    return p.x_dtype == 0 ? launch_few<float, __nv_bfloat16>(p, n_sm, st)
                          : launch_few<__nv_bfloat16, __nv_bfloat16>(p, n_sm, st);
}

}  // namespace moe
