// Matrix-vector products with 4-bit weights and group scales: y = W x for a
// dense weight matrix in HBM and a few tokens, on the library's int8 blocks.
//
//   y[t][r] = sum_b term(W block (r, b), x block (t, b)), block dots exact in
//   int32, Q4_0: d_w d_a sum_i (q_w,i - 8) q_a,i
//   Q4_K:  d_a (d sc_j sum_i q_w,i q_a,i - dmin m_j sum_i q_a,i)
//
// Weight layout (made at registration from the canonical blocks): a plane of
// codes, [rows][cols/32] x 16 bytes in Q4 order, then Q4_0: the binary16
// scales [rows][cols/32]; Q4_K: the 16 header bytes (d, dmin, 12 packed
// scale / min bytes) of every super-block [rows][cols/256].  18 bytes to 32
// weights either way, 16-byte aligned code loads.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kWarpsLin = 8;

// Canonical blocks -> planes.
__global__ void linear_repack_kernel(const uint8_t *__restrict__ src, uint8_t *__restrict__ dst, int fmt, size_t nblk) {
    for (size_t b = (size_t)blockIdx.x * blockDim.x + threadIdx.x; b < nblk; b += (size_t)gridDim.x * blockDim.x) {
        uint8_t *q = dst + 16 * b;
        if (fmt == kFmtQ4) {
            const uint8_t *s = src + 18 * b;
            for (int i = 0; i < 16; ++i) q[i] = s[2 + i];
            dst[16 * nblk + 2 * b] = s[0];
            dst[16 * nblk + 2 * b + 1] = s[1];
        } else {
            // sub-block j of a 144-byte super-block: 32 nibbles of chunk j / 2
            const int j = (int)(b & 7);
            const uint8_t *s = src + 144 * (b >> 3), *c = s + 16 + 32 * (j >> 1);
            const int sh = (j & 1) * 4;
            for (int i = 0; i < 16; ++i) q[i] = (uint8_t)(((c[i] >> sh) & 15) | (((c[i + 16] >> sh) & 15) << 4));
            dst[16 * nblk + 2 * b] = s[2 * j];
            dst[16 * nblk + 2 * b + 1] = s[2 * j + 1];
        }
    }
}

// Scale data of one weight block.
template <int FMT>
struct LinScale;
template <>
struct LinScale<kFmtQ4> {
    float s;
    __device__ __forceinline__ void load(const uint8_t *scales, size_t b) {
        s = __half2float(__ldcs((const __half *)scales + b));
    }
    __device__ __forceinline__ float term(int raw, float da, int sa) const {
        return (float)(raw - 8 * sa) * (s * da);
    }
    __device__ __forceinline__ unsigned bound() const { return __float_as_uint(fabsf(8.0f * s)); }
};
template <>
struct LinScale<kFmtQ4K> {
    float sc, mn;
    __device__ __forceinline__ void load(const uint8_t *scales, size_t b) {
        const uint4 h = __ldg((const uint4 *)scales + (b >> 3));
        const int j = (int)(b & 7), sh = 8 * (j & 3);
        const uint32_t a = h.y >> sh, m = h.z >> sh, x = h.w >> sh;
        const int s6 = j < 4 ? (a & 63) : ((x & 15) | (((a >> 6) & 3) << 4));
        const int m6 = j < 4 ? (m & 63) : (((x >> 4) & 15) | (((m >> 6) & 3) << 4));
        sc = __half2float(__ushort_as_half((unsigned short)(h.x & 0xffff))) * (float)s6;
        mn = __half2float(__ushort_as_half((unsigned short)(h.x >> 16))) * (float)m6;
    }
    __device__ __forceinline__ float term(int raw, float da, int sa) const {
        return da * (sc * (float)raw - mn * (float)sa);
    }
    __device__ __forceinline__ unsigned bound() const {
        return max(__float_as_uint(fabsf(mn)), __float_as_uint(fabsf(15.0f * sc - mn)));
    }
};

// Largest magnitude a block's weights can take, over the matrix, as binary32
// bits (NaN above infinity above all): *out, zero before.
template <int FMT>
__global__ void linear_max_kernel(const uint8_t *__restrict__ w, size_t nblk, unsigned *out) {
    unsigned m = 0;
    for (size_t b = (size_t)blockIdx.x * blockDim.x + threadIdx.x; b < nblk; b += (size_t)gridDim.x * blockDim.x) {
        LinScale<FMT> s;
        s.load(w + 16 * nblk, b);
        m = max(m, s.bound());
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) atomicMax(out, m);
}

// Sums V values a lane over the warp's lanes: halves the value set at each
// of the first log2(V) steps, so the total is V - 1 + 5 - log2(V) shuffles.
// Returns value `index` (by lane), complete.
template <int V>
__device__ __forceinline__ float reduce_scatter(float (&v)[V], int lane, int &index) {
    int off = 16;
    index = 0;
#pragma unroll
    for (int n = V; n > 1; n >>= 1) {
        const bool up = lane & off;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float send = up ? v[i] : v[i + n / 2], keep = up ? v[i + n / 2] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
        if (up) index += n / 2;
        off >>= 1;
    }
#pragma unroll
    for (; off > 0; off >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    return v[0];
}

// A warp computes R rows x TN tokens; lanes take every 32nd block of the rows.
// Shared memory: x codes as two planes of 16-byte halves [TN][nb], then
// {d, code sum} [TN][nb].
template <int FMT, int R, int TN>
__global__ void __launch_bounds__(32 * kWarpsLin) linear_matvec_kernel(LinearParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int nb = p.cols / kBlock, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int4 *x0 = (int4 *)smem, *x1 = x0 + TN * nb;
    BlockScale *xs = (BlockScale *)(x1 + TN * nb);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int t0 = blockIdx.y * TN, nt = min(TN, p.n_tokens - t0);
    // stage the tokens' codes (or quantize them): 8 lanes a block, 4 values a lane
    // (whole warps run every round: the shuffles need all lanes)
    for (int i0 = threadIdx.x - lane; i0 < TN * nb * 8; i0 += blockDim.x) {
        const int i = i0 + lane, w = i & 7, b = (i >> 3) % nb, t = (i >> 3) / nb;
        uint32_t code = 0;
        float dd = 0.0f;
        if (p.x) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (t < nt) v = *((const float4 *)(p.x + (size_t)(t0 + t) * p.cols) + b * 8 + w);
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
        } else if (t < nt) {
            code = *((const uint32_t *)(p.q + (size_t)(t0 + t) * p.cols) + b * 8 + w);
            dd = __half2float(p.d[(size_t)(t0 + t) * nb + b]);
        }
        int s = __dp4a((int)code, 0x01010101, 0);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (t >= TN) continue;  // past the last block
        ((uint32_t *)(w < 4 ? x0 : x1))[(t * nb + b) * 4 + (w & 3)] = code;
        if (w == 0) xs[t * nb + b] = BlockScale{dd, s};
    }
    __syncthreads();
    const uint8_t *scales = p.w + (size_t)p.rows * nb * 16;
    for (int r0 = (blockIdx.x * kWarpsLin + warp) * R; r0 < p.rows; r0 += gridDim.x * kWarpsLin * R) {
        float acc[R * TN];
#pragma unroll
        for (int i = 0; i < R * TN; ++i) acc[i] = 0.0f;
        for (int b = lane; b < nb; b += 32) {
            uint4 c[R];
            LinScale<FMT> sc[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const size_t blk = (size_t)min(r0 + r, p.rows - 1) * nb + b;
                c[r] = ld_weights((const uint4 *)p.w + blk);
                sc[r].load(scales, blk);
            }
#pragma unroll
            for (int t = 0; t < TN; ++t) {
                const int4 a0 = x0[t * nb + b], a1 = x1[t * nb + b];
                const BlockScale xa = xs[t * nb + b];
#pragma unroll
                for (int r = 0; r < R; ++r) acc[r * TN + t] += sc[r].term(q4_dot_raw(c[r], a0, a1), xa.d, xa.s);
            }
        }
        int i;
        const float v = reduce_scatter<R * TN>(acc, lane, i);
        const int r = i / TN, t = i % TN;
        if ((lane & (32 / (R * TN) - 1)) == 0 && r0 + r < p.rows && t < nt)
            p.y[(size_t)(t0 + t) * p.rows + r0 + r] = v;
    }
}

template <int FMT, int R, int TN>
int launch_mv(const LinearParams &p, int n_sm, cudaStream_t st) {
    auto kernel = linear_matvec_kernel<FMT, R, TN>;
    const size_t smem = (size_t)TN * (p.cols / kBlock) * (32 + sizeof(BlockScale));
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinearMaxSmem);
        if (e != cudaSuccess) return (int)e;
    }
    cudaLaunchConfig_t cfg{};
    const int per = kWarpsLin * R, fit = (int)std::max<size_t>(1, std::min<size_t>(8, 220 * 1024 / (smem + 1024)));
    cfg.gridDim = dim3((unsigned)std::min((p.rows + per - 1) / per, n_sm * fit), (unsigned)((p.n_tokens + TN - 1) / TN));
    cfg.blockDim = dim3(32 * kWarpsLin);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int FMT, int TN>
int launch_rows(const LinearParams &p, int n_sm, cudaStream_t st) {
    if (p.rows <= n_sm * kWarpsLin) return launch_mv<FMT, 1, TN>(p, n_sm, st);
    return launch_mv<FMT, 4, TN>(p, n_sm, st);
}

template <int FMT>
int launch_tokens(const LinearParams &p, int n_sm, cudaStream_t st) {
    // tokens a pass: what shared memory holds
    const size_t one = (size_t)(p.cols / kBlock) * (32 + sizeof(BlockScale));
    if (p.n_tokens >= 5 && 8 * one <= (size_t)kLinearMaxSmem) return launch_rows<FMT, 8>(p, n_sm, st);
    if (p.n_tokens >= 3 && 4 * one <= (size_t)kLinearMaxSmem) return launch_rows<FMT, 4>(p, n_sm, st);
    if (p.n_tokens >= 2 && 2 * one <= (size_t)kLinearMaxSmem) return launch_rows<FMT, 2>(p, n_sm, st);
    return launch_rows<FMT, 1>(p, n_sm, st);
}

}  // namespace

int launch_linear_repack(const uint8_t *src, uint8_t *dst, int fmt, size_t nblk, int n_sm, cudaStream_t st) {
    const unsigned g = (unsigned)std::min<size_t>((nblk + 255) / 256, (size_t)n_sm * 8);
    linear_repack_kernel<<<g, 256, 0, st>>>(src, dst, fmt, nblk);
    return (int)cudaGetLastError();
}

int launch_linear_max(const uint8_t *w, int fmt, size_t nblk, unsigned *out, int n_sm, cudaStream_t st) {
    const unsigned g = (unsigned)std::min<size_t>((nblk + 255) / 256, (size_t)n_sm * 8);
    if (fmt == kFmtQ4K)
        linear_max_kernel<kFmtQ4K><<<g, 256, 0, st>>>(w, nblk, out);
    else
        linear_max_kernel<kFmtQ4><<<g, 256, 0, st>>>(w, nblk, out);
    return (int)cudaGetLastError();
}

int launch_linear(const LinearParams &p, int n_sm, cudaStream_t st) {
    return p.fmt == kFmtQ4K ? launch_tokens<kFmtQ4K>(p, n_sm, st) : launch_tokens<kFmtQ4>(p, n_sm, st);
}

}  // namespace moe
