// y = W x of a dense layer with 4-bit weights and group scales, on the library's
// int8 blocks: registration, and the kernel of few tokens (batches:
// kernels_linear_gemm.cu).
//
//   y[t][r] = sum_b term(W block (r, b), x block (t, b)), block dots exact in
//   int32, Q4_0: d_w d_a sum_i (q_w,i - 8) q_a,i
//   Q4_K: d sc_j d_a sum_i q_w,i q_a,i - dmin m_j d_a sum_i q_a,i
//
// Bound: at one token the weights' one read from HBM: 65536 x 2048 (75.5 MB)
// 14.6 us = 5.2 TB/s, 0.76 of a copy's rate (Q4_K 15.5 us); 512 x 2048 2.3 us
// (latency).  With more tokens the time grows with the dots and the activations'
// shared-memory reads: 2 tokens 18.7 us, 3 26.3, 4 26.8 (Q4_K 29.5), where the
// tensor cores' path takes 45 (67); an earlier form of this kernel took 53 at 8
// tokens.
//
// Weight layout (made at registration): per 16 rows, per group of up to 8
// blocks: the codes [block][row] x 16 bytes in Q4 order, then the scales: Q4_0
// [block][g] x (binary16 d of rows g, g + 8); Q4_K [block][g] x bytes (sc, m of
// row g; of row g + 8), then [g] x (d, dmin of row g; of row g + 8).  18 (Q4_K
// 18.5) bytes to 32 weights.  16 lanes read 256 contiguous bytes of codes, and
// a lane keeps one row: its sum leaves the warp through one shuffle.
#include <algorithm>

#include "kernels.h"
#include "linear.cuh"

namespace moe {
namespace {

// ---- registration -------------------------------------------------------------
// One thread a (row of the padded matrix, block).
__global__ void linear_repack_kernel(const uint8_t *__restrict__ src, uint8_t *__restrict__ dst, int fmt, int rows,
                                     int nb) {
    const size_t n = (size_t)((rows + 15) / 16) * 16 * nb;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x) {
        const size_t row = i / nb;
        const int b = (int)(i % nb), r = (int)(row & 15), g = r & 7, up = r >> 3, b0 = b / kKB * kKB, bi = b - b0;
        const int cnt = min(kKB, nb - b0);
        uint8_t *grp = dst + (row >> 4) * tile_bytes(fmt, nb) +
                       (fmt == kFmtQ4K ? (size_t)(b0 / kKB) * group_bytes(fmt, kKB) : (size_t)b0 * kARec);
        uint8_t *sc = grp + cnt * 256 + bi * 32 + g * 4 + up * 2;
        uint32_t w[4] = {0, 0, 0, 0};
        uint8_t s0 = 0, s1 = 0;
        const bool on = row < (size_t)rows;
        if (fmt == kFmtQ4) {
            const uint8_t *s = src + 18 * (row * nb + b);
            if (on) {
                for (int j = 0; j < 16; ++j) w[j >> 2] |= (uint32_t)s[2 + j] << (8 * (j & 3));
                s0 = s[0];
                s1 = s[1];
            }
        } else {
            const uint8_t *s = src + 144 * ((row * nb + b) >> 3);
            uint8_t *dm = grp + kKB * kARec + g * 8 + up * 4;
            if (on) {
                const uint8_t *c = s + 16 + 32 * (bi >> 1), *p = s + 4;
                const int sh = (bi & 1) * 4;
                for (int j = 0; j < 16; ++j)
                    w[j >> 2] |= (uint32_t)(((c[j] >> sh) & 15) | (((c[j + 16] >> sh) & 15) << 4)) << (8 * (j & 3));
                s0 = bi < 4 ? (p[bi] & 63) : ((p[bi + 4] & 15) | ((p[bi - 4] >> 6) << 4));
                s1 = bi < 4 ? (p[bi + 4] & 63) : ((p[bi + 4] >> 4) | ((p[bi] >> 6) << 4));
            }
            if (bi == 0)
                for (int j = 0; j < 4; ++j) dm[j] = on ? s[j] : 0;
        }
        sc[0] = s0;
        sc[1] = s1;
        *(uint4 *)(grp + bi * 256 + r * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ---- activations --------------------------------------------------------------
// Word w (elements 4w..4w+3) of token t's block b as it is in memory: four fp32
// values, or the code word and the scale.
struct RawWord {
    float4 v;
    __device__ __forceinline__ void load(const LinearParams &p, size_t t, int b, int w, bool on) {
        v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (!on) return;
        if (p.x) {
            v = __ldcg((const float4 *)(p.x + t * p.cols) + b * 8 + w);
        } else {
            v.x = __uint_as_float(__ldcg((const uint32_t *)(p.q + t * p.cols) + b * 8 + w));
            v.y = __half2float(__ushort_as_half(__ldcg((const unsigned short *)p.d + t * (p.cols / kBlock) + b)));
        }
    }
    // The code word, the scale and, over the block's 8 lanes, the code sum.
    // All lanes of a warp call.
    __device__ __forceinline__ void finish(bool fp, uint32_t &code, float &dd, int &sum) const {
        if (fp) {
            code = 0;
            unsigned m = max(max(__float_as_uint(fabsf(v.x)), __float_as_uint(fabsf(v.y))),
                             max(__float_as_uint(fabsf(v.z)), __float_as_uint(fabsf(v.w))));
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            dd = __half2float(__float2half_rn(__uint_as_float(m) / 127.0f));
            const float e[4] = {v.x, v.y, v.z, v.w};
            if (dd != 0.0f)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    code |= ((uint32_t)(int)fminf(fmaxf(rintf(e[j] / dd), -127.0f), 127.0f) & 255u) << (8 * j);
        } else {
            code = __float_as_uint(v.x);
            dd = v.y;
        }
        sum = __dp4a((int)code, 0x01010101, 0);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
};

// ---- up to four tokens ------------------------------------------------------------
// A lane owns a row of the tile and the blocks of its half warp; the CTA's
// warps take the tile's block pairs in turn, kFly pairs in flight each, the
// next tile's first ones requested before this tile's sums are joined.
constexpr int kVecWarps = 8, kFly = 4;

template <int FMT>
struct VBlock {
    uint4 c;
    uint32_t s, dm;  // Q4_0: d; Q4_K: (sc, m) and (d, dmin)
    __device__ __forceinline__ void load(const uint8_t *tile, int nb, int b, int r) {
        const int n = min(kKB, nb - b / kKB * kKB), bi = b % kKB;
        const uint8_t *grp = tile + (size_t)(b / kKB) * group_bytes(FMT, kKB);
        c = ld_weights((const uint4 *)(grp + bi * 256 + r * 16));
        s = __ldcs((const unsigned short *)(grp + n * 256 + bi * 32) + (r & 7) * 2 + (r >> 3));
        if (FMT == kFmtQ4K) dm = __ldg((const uint32_t *)(grp + kKB * kARec) + (r & 7) * 2 + (r >> 3));
    }
    // the block's scale and (Q4_K) minus its min
    __device__ __forceinline__ float2 scale() const {
        if (FMT == kFmtQ4) return make_float2(__half2float(__ushort_as_half((unsigned short)s)), 0.0f);
        const float2 d = __half22float2(*(const __half2 *)&dm);
        return make_float2(d.x * (float)(s & 255), -d.y * (float)(s >> 8));
    }
};

// The dot counts up from the bits of 1.5 x 2^23 (less 8 sum q_a for Q4_0): its
// integer, below 2^17, is that float's offset, and no conversion is needed.
constexpr int kMagic = 0x4B400000;
constexpr float kMagicF = 12582912.0f;

// acc += the block's term.  x.s: Q4_0 kMagic - 8 sum q_a; Q4_K sum q_a.
template <int FMT>
__device__ __forceinline__ float add_term(const uint4 &c, const float2 &w, const int4 &a0, const int4 &a1,
                                          const BlockScale &x, float acc) {
    const uint32_t m = 0x0F0F0F0Fu;
    int s = FMT == kFmtQ4 ? x.s : kMagic;
    s = __dp4a((int)(c.x & m), a0.x, s);
    s = __dp4a((int)(c.y & m), a0.y, s);
    s = __dp4a((int)(c.z & m), a0.z, s);
    s = __dp4a((int)(c.w & m), a0.w, s);
    s = __dp4a((int)((c.x >> 4) & m), a1.x, s);
    s = __dp4a((int)((c.y >> 4) & m), a1.y, s);
    s = __dp4a((int)((c.z >> 4) & m), a1.z, s);
    s = __dp4a((int)((c.w >> 4) & m), a1.w, s);
    const float dot = __int_as_float(s) - kMagicF;
    if (FMT == kFmtQ4) return fmaf(dot, w.x * x.d, acc);
    acc = fmaf(dot * x.d, w.x, acc);
    return fmaf((float)x.s * x.d, w.y, acc);
}

template <int FMT, int TN, int kBatch>
__global__ void __launch_bounds__(kVecWarps * 32, TN > 2 ? 3 : 4) linear_vec_kernel(const __grid_constant__ LinearParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][kVecWarps][TN][16];
    const int nb = p.cols / kBlock, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane & 15;
    int4 *x0 = (int4 *)smem, *x1 = x0 + TN * nb;  // codes: elements 0..15 and 16..31 of a block, [TN][nb]
    BlockScale *xs = (BlockScale *)(x1 + TN * nb);
    const int rt_n = (p.rows + 15) / 16, first = 2 * warp + (lane >> 4);
    const int t0 = blockIdx.y * TN, nt = min(TN, p.n_tokens - t0);
    const size_t rt_bytes = tile_bytes(FMT, nb);
    VBlock<FMT> w[kFly];
    auto fetch = [&](int tile, int b0) {
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            const int b = b0 + i * 2 * kVecWarps;
            if (b < nb) w[i].load(p.w + tile * rt_bytes, nb, b, r);
        }
    };
    // the weights are the context's own: requested before the wait
    if ((int)blockIdx.x < rt_n) fetch(blockIdx.x, first);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    // the activations: 8 lanes a block, 4 values a lane, kBatch rounds' loads in
    // flight (whole warps run every round)
    for (int i0 = warp * 32; i0 < TN * nb * 8; i0 += kBatch * kVecWarps * 32) {
        RawWord raw[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + k * kVecWarps * 32 + lane, tb = i >> 3, t = TN > 1 ? tb / nb : 0;
            raw[k].load(p, t0 + t, tb - t * nb, i & 7, tb < nt * nb);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + k * kVecWarps * 32 + lane, q = i & 7, tb = i >> 3;
            uint32_t code;
            float dd;
            int sum;
            raw[k].finish(p.x != nullptr, code, dd, sum);
            if (tb >= TN * nb) continue;
            ((uint32_t *)(q < 4 ? x0 : x1))[tb * 4 + (q & 3)] = code;
            if (q == 0) xs[tb] = BlockScale{dd, FMT == kFmtQ4 ? kMagic - 8 * sum : sum};
        }
    }
    __syncthreads();
    int turn = 0;
    for (int tile = blockIdx.x; tile < rt_n; tile += gridDim.x, turn ^= 1) {
        float acc[TN];
#pragma unroll
        for (int t = 0; t < TN; ++t) acc[t] = 0.0f;
        for (int b0 = first; b0 - (lane >> 4) < nb; b0 += kFly * 2 * kVecWarps) {
            if (b0 != first) fetch(tile, b0);
#pragma unroll
            for (int i = 0; i < kFly; ++i) {
                const int b = b0 + i * 2 * kVecWarps;
                if (b < nb) {
                    const float2 sc = w[i].scale();
#pragma unroll
                    for (int t = 0; t < TN; ++t)
                        acc[t] = add_term<FMT>(w[i].c, sc, x0[t * nb + b], x1[t * nb + b], xs[t * nb + b], acc[t]);
                }
            }
        }
        if (tile + (int)gridDim.x < rt_n) fetch(tile + gridDim.x, first);
#pragma unroll
        for (int t = 0; t < TN; ++t) {
            acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], 16);
            if (lane < 16) red[turn][warp][t][r] = acc[t];
        }
        __syncthreads();
        // (the other buffer of red is free: its readers have passed this barrier)
        if (threadIdx.x < 16 * TN) {
            const int t = threadIdx.x / 16, row = tile * 16 + threadIdx.x % 16;
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < kVecWarps; ++k) v += red[turn][k][t][threadIdx.x % 16];
            if (row < p.rows && t < nt) p.y[(size_t)(t0 + t) * p.rows + row] = v;
        }
    }
}

// Largest magnitude a block's weights can take, over the matrix, as binary32
// bits (NaN above infinity above all): *out, zero before.  Q4_K: also the rows'
// powers of two, which bring a row's largest magnitude to [2^14, 2^15) (1 for a
// row of zeros).  A warp a row.
template <int FMT>
__global__ void linear_max_kernel(const uint8_t *w, int rows, int nb, float *row_scale, unsigned *out) {
    const int lane = threadIdx.x & 31, rt_n = (rows + 15) / 16;
    const size_t n = (size_t)(rows + kScaleRows - 1) / kScaleRows * kScaleRows;
    unsigned top = 0;
    for (size_t row = ((size_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; row < n;
         row += (size_t)gridDim.x * blockDim.x >> 5) {
        unsigned m = 0;
        if (row >> 4 < (size_t)rt_n)
            for (int b = lane; b < nb; b += 32) {
                VBlock<FMT> v;
                v.load(w + (row >> 4) * tile_bytes(FMT, nb), nb, b, (int)(row & 15));
                const float2 s = v.scale();
                m = max(m, FMT == kFmtQ4
                               ? __float_as_uint(fabsf(8.0f * s.x))
                               : max(__float_as_uint(fabsf(s.y)), __float_as_uint(fabsf(fmaf(15.0f, s.x, s.y)))));
            }
        m = __reduce_max_sync(0xffffffffu, m);
        top = max(top, m);
        // (magnitudes are multiples of 2^-24 and below 2^27: the exponents stay in range; a layer with
        // infinities or NaN has no use for them)
        if (FMT == kFmtQ4K && lane == 0)
            row_scale[row] = m && m < 0x7f800000u ? __uint_as_float((127u + 127u + 14u - (m >> 23)) << 23) : 1.0f;
    }
    if (lane == 0) atomicMax(out, top);
}

// ---- launch ---------------------------------------------------------------------
template <int FMT, int TN, int BATCH>
int launch_batch(const LinearParams &p, int n_sm, cudaStream_t st) {
    auto kernel = linear_vec_kernel<FMT, TN, BATCH>;
    static bool done[64];  // the shared memory limit, raised once a device
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinearSmem);
        if (e != cudaSuccess) return (int)e;
        if (dev >= 0 && dev < 64) done[dev] = true;
    }
    const size_t smem = (size_t)TN * (p.cols / kBlock) * (32 + sizeof(BlockScale));
    const int fit = (int)std::max<size_t>(1, std::min<size_t>(TN > 2 ? 3 : 4, 220 * 1024 / (smem + 10 * 1024)));
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kVecWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // a grid has at most 65535 groups of tokens
    const size_t total = p.n_tokens, most = 65535 * TN;
    for (size_t t = 0; t < total; t += most) {
        LinearParams part = p;
        part.n_tokens = (int)std::min(total - t, most);
        if (p.x) part.x += t * p.cols;
        if (p.q) part.q += t * p.cols, part.d += t * (p.cols / kBlock);
        part.y += t * p.rows;
        cfg.gridDim = dim3((unsigned)std::min((p.rows + 15) / 16, n_sm * fit), (unsigned)((part.n_tokens + TN - 1) / TN));
        const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, part);
        if (e != cudaSuccess) return (int)e;
    }
    return 0;
}

template <int FMT, int TN>
int launch_vec(const LinearParams &p, int n_sm, cudaStream_t st) {
    // rounds of the activations' staging: 1024 values each
    return TN * p.cols > 2048 ? launch_batch<FMT, TN, 4>(p, n_sm, st) : launch_batch<FMT, TN, 2>(p, n_sm, st);
}

template <int FMT>
int launch_fmt(const LinearParams &p, int n_sm, cudaStream_t st) {
    // two tokens a pass over the weights where their activations fit
    const size_t one = (size_t)(p.cols / kBlock) * (32 + sizeof(BlockScale));
    if (p.n_tokens >= 3 && 4 * one <= (size_t)kLinearSmem) return launch_vec<FMT, 4>(p, n_sm, st);
    if (p.n_tokens >= 2 && 2 * one <= (size_t)kLinearSmem) return launch_vec<FMT, 2>(p, n_sm, st);
    return launch_vec<FMT, 1>(p, n_sm, st);
}

}  // namespace

size_t linear_weight_bytes(int fmt, int rows, int cols) {
    const size_t scales = fmt == kFmtQ4K ? (size_t)(rows + kScaleRows - 1) / kScaleRows * kScaleRows * 4 : 0;
    return row_scale_offset(fmt, rows, cols / kBlock) + scales;
}

int launch_linear_repack(const uint8_t *src, uint8_t *dst, int fmt, int rows, int cols, int n_sm, cudaStream_t st) {
    const size_t n = (size_t)((rows + 15) / 16) * 16 * (cols / kBlock);
    const unsigned g = (unsigned)std::min<size_t>((n + 255) / 256, (size_t)n_sm * 8);
    linear_repack_kernel<<<g, 256, 0, st>>>(src, dst, fmt, rows, cols / kBlock);
    return (int)cudaGetLastError();
}

int launch_linear_max(uint8_t *w, int fmt, int rows, int cols, unsigned *out, int n_sm, cudaStream_t st) {
    const int nb = cols / kBlock;
    const unsigned g = (unsigned)std::min(rows / 8 + kScaleRows / 8, n_sm * 8);  // 8 rows a CTA
    if (fmt == kFmtQ4K)
        linear_max_kernel<kFmtQ4K><<<g, 256, 0, st>>>(w, rows, nb, (float *)(w + row_scale_offset(fmt, rows, nb)), out);
    else
        linear_max_kernel<kFmtQ4><<<g, 256, 0, st>>>(w, rows, nb, nullptr, out);
    return (int)cudaGetLastError();
}

int launch_linear(const LinearParams &p, int n_sm, cudaStream_t st) {
    return p.fmt == kFmtQ4K ? launch_fmt<kFmtQ4K>(p, n_sm, st) : launch_fmt<kFmtQ4>(p, n_sm, st);
}

}  // namespace moe
