// y = W x of a dense layer with 4-bit weights and group scales, from one token
// to prompt chunks, on the library's int8 blocks.
//
//   y[t][r] = sum_b term(W block (r, b), x block (t, b)), block dots exact,
//   Q4_0: d_w d_a sum_i (q_w,i - 8) q_a,i
//   Q4_K: d sc_j d_a sum_i q_w,i q_a,i - dmin m_j d_a sum_i q_a,i
//
// Block dots on the tensor cores, exactly: a low nibble under the binary16
// exponent 0x64 is 1024 + q, a high one in its place 1024 + 16 q; the codes of
// the low nibbles' elements (0..15) are binary16 integers, those of the high
// ones' (16..31) sixteenths, and the two m16n8k16 products of a block start
// from minus what the 1024s (and Q4_0's offset 8) add, -(1024 S_lo + 64 S_hi +
// 8 S) of the code sums, so that they end at the block's dot.  Every partial
// sum is a multiple of 1 below 2^24 (64 a + a q and the like), which fp32 holds.  The sums stay in registers and their scaling
// costs two packed fp32 operations for two sums.  That is why this runs on
// mma.sync (594 TFLOP/s of f16 measured; s8 151, dp4a 149, e4m3 lowered to
// f16): tcgen05 leaves its sums in TMEM, where reading every block's sums back
// bounds the experts' GEMM at 0.07 of the peak, and folding the scales into two
// binary16 parts of each operand (three tcgen05 products a step, weights
// through TMEM) measured 63 us for 4096 x 4096 at 512 tokens, with larger
// errors.
//
// One and two tokens take dp4a on whole blocks instead: 15 warp instructions
// for 16 x 32 weights and a token against 40 for any 8 tokens.
//
// Weight layout (made at registration): per 16 rows, per group of up to 8
// blocks: the codes [block][row] x 16 bytes in Q4 order, then the scales: Q4_0
// [block][g] x (binary16 d of rows g, g + 8); Q4_K [block][g] x bytes (sc, m of
// row g; of row g + 8), then [g] x (d, dmin of row g; of row g + 8).  18 (Q4_K
// 18.5) bytes to 32 weights, and any run of groups of 16 rows is one contiguous
// copy.  Lane 4g + t of a product holds word t of rows g and g + 8: elements
// 4t + (0, 2), 16 + 4t + (0, 2), 4t + (1, 3), 16 + 4t + (1, 3) as its four
// pairs of K; the sums do not mind the order.
//
// Activation layout of the products: per 8 tokens, per block: [lane] x 16
// bytes (lane 4c + t: token c's codes in binary16, in the same order), then for
// tokens 2t, 2t + 1: [t] x 16 what their products start from, twice; [t] x 8
// d_a; Q4_K: [t] x 8 d_a times the code sum.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace moe {
namespace {

using namespace gemm;

constexpr int kKB = 8;            // blocks of a group: a pipeline stage
constexpr int kARec = 16 * 18;    // bytes of 16 rows of a Q4_0 block
// bytes of 8 tokens of a block: codes, starting values, scales (Q4_K: and sums)
__host__ __device__ constexpr int act_bytes(int fmt) { return 512 + 64 + 32 + (fmt == kFmtQ4K ? 32 : 0); }

// bytes of a group of n blocks of 16 rows, and of all nb
__host__ __device__ constexpr int group_bytes(int fmt, int n) { return n * kARec + (fmt == kFmtQ4K ? 64 : 0); }
__host__ __device__ inline size_t tile_bytes(int fmt, int nb) {
    return (size_t)nb * kARec + (fmt == kFmtQ4K ? (size_t)(nb / kKB) * 64 : 0);
}

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
// Word w (elements 4w..4w+3) of token t's block b: the code word, the scale
// and, over the 4 lanes of the block's half, the code sum.  All lanes of a warp
// call.
__device__ __forceinline__ void code_word(const LinearParams &p, size_t t, int b, int w, bool on, uint32_t &code,
                                          float &dd, int &sum) {
    code = 0;
    dd = 0.0f;
    if (p.x) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (on) v = __ldcg((const float4 *)(p.x + t * p.cols) + b * 8 + w);
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
    } else if (on) {
        code = __ldcg((const uint32_t *)(p.q + t * p.cols) + b * 8 + w);
        dd = __half2float(__ushort_as_half(__ldcg((const unsigned short *)p.d + t * (p.cols / kBlock) + b)));
    }
    sum = __dp4a((int)code, 0x01010101, 0);
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
}

// ... into the record of its block, token column c of 8 (all lanes call).
__device__ __forceinline__ void put_word(uint8_t *rec, int c, int w, uint32_t code, float dd, int sum, int fmt) {
    // codes + 128 under the binary16 exponent 0x64: 1152 + q; bytes (0, 2), (1, 3)
    const uint32_t u = code ^ 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const __half2 unit = w < 4 ? __float2half2_rn(1.0f) : __float2half2_rn(0.0625f);
    uint32_t h[2] = {__byte_perm(u, 0x64646464u, 0x4240), __byte_perm(u, 0x64646464u, 0x4341)};
#pragma unroll
    for (int i = 0; i < 2; ++i) *(__half2 *)&h[i] = __hmul2(__hsub2(*(__half2 *)&h[i], off), unit);
    uint32_t *f = (uint32_t *)(rec + (4 * c + (w & 3)) * 16) + (w >> 2);
    f[0] = h[0];
    f[2] = h[1];
    const int high = __shfl_down_sync(0xffffffffu, sum, 4);
    if (w == 0) {
        const int all = sum + high;
        const float start = -(float)(1024 * sum + 64 * high + (fmt == kFmtQ4K ? 0 : 8 * all));
        float *st = (float *)(rec + 512 + (c >> 1) * 16) + (c & 1);
        st[0] = st[2] = start;
        *((float *)(rec + 576 + (c >> 1) * 8) + (c & 1)) = dd;
        if (fmt == kFmtQ4K) *((float *)(rec + 608 + (c >> 1) * 8) + (c & 1)) = dd * (float)all;
    }
}

// Records of 8 tokens (blockIdx.x) x 4 blocks (blockIdx.y) to the workspace;
// tokens past the last are zeros.
__global__ void __launch_bounds__(256) linear_prepare_kernel(LinearParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ __align__(16) uint8_t rec[4 * act_bytes(kFmtQ4K)];
    const int bytes = act_bytes(p.fmt);
    const int nb = p.cols / kBlock, w = threadIdx.x & 7, c = (threadIdx.x >> 3) & 7, bi = threadIdx.x >> 6;
    const int b = blockIdx.y * 4 + bi, t = blockIdx.x * 8 + c, n = min(4, nb - (int)blockIdx.y * 4);
    uint32_t code;
    float dd;
    int sum;
    code_word(p, t, b, w, t < p.n_tokens && b < nb, code, dd, sum);
    put_word(rec + bi * bytes, c, w, code, dd, sum, p.fmt);
    __syncthreads();
    uint4 *out = (uint4 *)(p.ws + ((size_t)blockIdx.x * nb + blockIdx.y * 4) * bytes);
    for (int i = threadIdx.x; i < n * (bytes / 16); i += 256) out[i] = ((const uint4 *)rec)[i];
}

// ---- the product ----------------------------------------------------------------
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// d = a b + c on the 16 x 8 tile, binary16 operands, K = 16
__device__ __forceinline__ void mma_f16_sync(float (&d)[4], const uint32_t *a, uint32_t b0, uint32_t b1, float c0,
                                             float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// packed fp32 pairs
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ float2 un2(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}

// A lane's share of a block's weights: the operand and rows g, g + 8's scales.
template <int FMT>
struct WFrag {
    uint32_t a[8];  // both products' operands
    F2 s[2], m[2];  // scale of each row, twice; Q4_K: minus its min, twice
    __device__ __forceinline__ void load(const uint8_t *grp, int n, int b, int lane) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t c = *(const uint32_t *)(grp + b * 256 + r * 128 + lane * 4);
            a[r] = (c & 0x000F000Fu) | 0x64006400u;
            a[2 + r] = (c & 0x00F000F0u) | 0x64006400u;
            a[4 + r] = ((c >> 8) & 0x000F000Fu) | 0x64006400u;
            a[6 + r] = ((c >> 8) & 0x00F000F0u) | 0x64006400u;
        }
        const int g = lane >> 2;
        const uint32_t w = *(const uint32_t *)(grp + n * 256 + b * 32 + g * 4);
        if (FMT == kFmtQ4) {
            const float2 d = __half22float2(*(const __half2 *)&w);
            s[0] = f2(d.x, d.x);
            s[1] = f2(d.y, d.y);
        } else {
            const uint2 dm = *(const uint2 *)(grp + kKB * kARec + g * 8);
            // bytes under the binary16 exponent 0x64: 1024 + value
            const uint32_t b0 = __byte_perm(w, 0x64646464u, 0x5150), b1 = __byte_perm(w, 0x64646464u, 0x5352);
            const float2 d0 = __half22float2(*(const __half2 *)&dm.x), d1 = __half22float2(*(const __half2 *)&dm.y);
            const float2 v0 = __half22float2(*(const __half2 *)&b0), v1 = __half22float2(*(const __half2 *)&b1);
            const float s0 = d0.x * (v0.x - 1024.0f), m0 = -d0.y * (v0.y - 1024.0f);
            const float s1 = d1.x * (v1.x - 1024.0f), m1 = -d1.y * (v1.y - 1024.0f);
            s[0] = f2(s0, s0);
            m[0] = f2(m0, m0);
            s[1] = f2(s1, s1);
            m[1] = f2(m1, m1);
        }
    }
};

constexpr int kNW = 16;  // warps of a CTA

// CTA tile: wr x MT x 16 rows, WC x NT x 8 tokens; the warps split the rows wr
// ways, the tokens WC ways, the stages of a tile ws ways and the blocks of a
// stage wb ways.  CTAs walk the tiles (token tiles innermost: they share the
// weights in L2) through a ring of stages of one group each; a warp that is
// done with a stage requests the one that takes its place.  The ring's length
// is a multiple of ws, so that a slot always belongs to the same warps: they
// see every phase of its barriers in turn.  RES: the records of all blocks stay in shared memory
// (one token tile), else a stage brings its own.
template <int FMT, int MT, int NT, int WC, bool RES>
__global__ void __launch_bounds__(kNW * 32, 1) linear_kernel(const __grid_constant__ LinearParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int wr_n = p.wr, wk_n = kNW / (WC * wr_n), ws_n = p.ws_n, wb_n = wk_n / ws_n, nb = p.cols / kBlock, ng = (nb + kKB - 1) / kKB;
    constexpr int NTC = NT * WC, GB = group_bytes(FMT, kKB), BST = kKB * act_bytes(FMT);
    const int a_stage = wr_n * MT * GB, stage = a_stage + (RES ? 0 : NTC * BST);
    uint8_t *resident = smem + p.stages * stage;
    float4 *red = (float4 *)(resident + (RES ? (size_t)NTC * nb * act_bytes(FMT) : 0));
    uint64_t *bars = (uint64_t *)(red + (wk_n > 1 ? kNW / 2 * MT * NT * 32 : 0));
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * p.stages, bfull = empty0 + 8 * p.stages;
    volatile int *abort_flag = (volatile int *)(bars + 2 * p.stages + 1);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, WC * wr_n * wb_n);
        }
        mbar_init(bfull, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    const int rt_n = (p.rows + 15) / 16, tile_rt = wr_n * MT, ntt = (p.n_tokens + 8 * NTC - 1) / (8 * NTC);
    const int total = ((rt_n + tile_rt - 1) / tile_rt) * ntt, nt_n = (p.n_tokens + 7) / 8;
    const size_t rt_bytes = tile_bytes(FMT, nb);
    const int n_it = ((total - 1 - (int)blockIdx.x) / (int)gridDim.x + 1) * ng;

    // Request stage j: lanes 0..tile_rt-1 a row tile's group each, lanes
    // 0..NTC-1 the tokens' records of the group.  The weights are the context's
    // own; the records are the preceding kernel's (part: 1 weights, 2 records).
    auto request = [&](int j, int part) {
        const int t = blockIdx.x + j / ng * gridDim.x, g = j % ng, slot = j % p.stages, n = min(kKB, nb - g * kKB);
        const int rt0 = t / ntt * tile_rt, n_rt = min(tile_rt, rt_n - rt0);
        const int nt0 = t % ntt * NTC, n_nt = RES ? 0 : min(NTC, nt_n - nt0);
        const uint32_t full = full0 + 8 * slot, dst = smem_u32(smem + slot * stage);
        if (part & 1) {
            bool ok = true;
            if (lane == 0) {
                ok = mbar_wait(empty0 + 8 * slot, ((uint32_t)(j / p.stages) & 1u) ^ 1u, abort_flag, p.error, 2);
                if (ok) mbar_arrive_tx(full, (uint32_t)(n_rt * group_bytes(FMT, n) + n_nt * n * act_bytes(FMT)));
            }
            if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) return;
            if (lane < n_rt)
                bulk_load(dst + lane * GB, p.w + (size_t)(rt0 + lane) * rt_bytes + (size_t)g * GB, group_bytes(FMT, n),
                          full);
        }
        if ((part & 2) && lane < n_nt)
            bulk_load(dst + a_stage + lane * BST, p.ws + ((size_t)(nt0 + lane) * nb + g * kKB) * act_bytes(FMT),
                      (uint32_t)(n * act_bytes(FMT)), full);
    };
    if (warp == 0) {
        const int first = min(p.stages, n_it);
        for (int j = 0; j < first; ++j) request(j, 1);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;");
        if (RES) {
            const int n = min(NTC, nt_n);
            if (lane == 0) mbar_arrive_tx(bfull, (uint32_t)(n * nb * act_bytes(FMT)));
            __syncwarp();
            if (lane < n)
                bulk_load(smem_u32(resident + (size_t)lane * nb * act_bytes(FMT)), p.ws + (size_t)lane * nb * act_bytes(FMT),
                          (uint32_t)(nb * act_bytes(FMT)), bfull);
        }
        for (int j = 0; j < first; ++j) request(j, 2);
    }
    // a wait that expires leaves garbage and an error bit; the warp goes on, so
    // that the others' barriers complete
    const int wc = warp % WC, wr = warp / WC % wr_n, wk = warp / (WC * wr_n);
    const int ws = wk % ws_n, wb = wk / ws_n;
    if (RES) mbar_wait(bfull, 0, abort_flag, p.error, 4);
    int it = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        F2 acc[MT][NT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = f2(0.0f, 0.0f);
        for (int g = 0; g < ng; ++g, ++it) {
            if (it % ws_n != ws) continue;
            const int slot = it % p.stages, n = min(kKB, nb - g * kKB);
            mbar_wait(full0 + 8 * slot, (uint32_t)(it / p.stages) & 1u, abort_flag, p.error, 4);
            const uint8_t *ga = smem + slot * stage + wr * MT * GB;
            const uint8_t *gb = RES ? resident + (size_t)g * kKB * act_bytes(FMT) : smem + slot * stage + a_stage + wc * NT * BST;
            const size_t b_tile = RES ? (size_t)nb * act_bytes(FMT) : BST;
            // several blocks at once where one has few products to hide its latency
            constexpr int kUnroll = MT * NT <= 2 ? 4 : MT * NT <= 4 ? 2 : 1;
#pragma unroll kUnroll
            for (int b = wb; b < n; b += wb_n) {
                WFrag<FMT> wf[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) wf[m].load(ga + m * GB, n, b, lane);
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    const uint8_t *rec = gb + c * b_tile + b * act_bytes(FMT);
                    const uint4 x = *(const uint4 *)(rec + lane * 16);
                    const float4 st = *(const float4 *)(rec + 512 + (lane & 3) * 16);
                    const float2 dv = *(const float2 *)(rec + 576 + (lane & 3) * 8);
                    const F2 da = f2(dv.x, dv.y);
                    float d[MT][4];
#pragma unroll
                    for (int m = 0; m < MT; ++m) mma_f16_sync(d[m], wf[m].a, x.x, x.y, st.x, st.y, st.z, st.w);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        mma_f16_sync(d[m], wf[m].a + 4, x.z, x.w, d[m][0], d[m][1], d[m][2], d[m][3]);
                    F2 e = da;
                    if (FMT == kFmtQ4K) {
                        const float2 ev = *(const float2 *)(rec + 608 + (lane & 3) * 8);
                        e = f2(ev.x, ev.y);
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const F2 v = mul2(f2(d[m][2 * h], d[m][2 * h + 1]), da);
                            acc[m][c][h] = fma2(wf[m].s[h], v, acc[m][c][h]);
                            if (FMT == kFmtQ4K) acc[m][c][h] = fma2(wf[m].m[h], e, acc[m][c][h]);
                        }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * slot);
            if ((wb * wr_n + wr) * WC + wc == it / ws_n % (wb_n * wr_n * WC) && it + p.stages < n_it) request(it + p.stages, 3);
        }
        // join the warps of one row and token share: the upper half of them
        // hands its sums to the lower half, until one is left
        for (int half = wk_n / 2; half > 0; half /= 2) {
            float4 *r = red + ((warp - (wk >= half ? half * wr_n * WC : 0)) * MT * NT) * 32 + lane;
            if (wk >= half && wk < 2 * half) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        const float2 u = un2(acc[m][c][0]), v = un2(acc[m][c][1]);
                        r[(m * NT + c) * 32] = make_float4(u.x, u.y, v.x, v.y);
                    }
            }
            __syncthreads();
            if (wk < half) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        const float4 o = r[(m * NT + c) * 32];
                        const float2 u = un2(acc[m][c][0]), v = un2(acc[m][c][1]);
                        acc[m][c][0] = f2(u.x + o.x, u.y + o.y);
                        acc[m][c][1] = f2(v.x + o.z, v.y + o.w);
                    }
            }
            __syncthreads();
        }
        if (wk > 0) continue;
        // lane 4g + q: rows g, g + 8 of a 16-row tile, tokens 2q, 2q + 1
        const int row0 = (t / ntt * tile_rt + wr * MT) * 16 + (lane >> 2);
        const int tok0 = (t % ntt * NTC + wc * NT) * 8 + (lane & 3) * 2;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = row0 + m * 16 + h * 8, tok = tok0 + c * 8;
                    const float2 v = un2(acc[m][c][h]);
                    if (row < p.rows && tok < p.n_tokens) p.y[(size_t)tok * p.rows + row] = v.x;
                    if (row < p.rows && tok + 1 < p.n_tokens) p.y[(size_t)(tok + 1) * p.rows + row] = v.y;
                }
    }
    // after an abort, give the copies in flight a bounded time (about 10 ms) to land
    __syncthreads();
    if (*abort_flag) {
        const long long t0 = clock64();
        while (clock64() - t0 < 20000000ll) {
        }
    }
}

// ---- one and two tokens -----------------------------------------------------------
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
    // acc += the block's term: raw = sum q_w q_a, the activations' scale and code sum
    __device__ __forceinline__ float term(int raw, const BlockScale &x, float acc) const {
        if (FMT == kFmtQ4)
            return fmaf((float)(raw - 8 * x.s), __half2float(__ushort_as_half((unsigned short)s)) * x.d, acc);
        const float2 d = __half22float2(*(const __half2 *)&dm);
        acc = fmaf(d.x * (float)(s & 255), x.d * (float)raw, acc);
        return fmaf(-d.y * (float)(s >> 8), x.d * (float)x.s, acc);
    }
};

template <int FMT, int TN>
__global__ void __launch_bounds__(kVecWarps * 32) linear_vec_kernel(const __grid_constant__ LinearParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][kVecWarps][TN][16];
    const int nb = p.cols / kBlock, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane & 15;
    int4 *x0 = (int4 *)smem, *x1 = x0 + TN * nb;  // codes: elements 0..15 and 16..31 of a block, [TN][nb]
    BlockScale *xs = (BlockScale *)(x1 + TN * nb);
    const int rt_n = (p.rows + 15) / 16, first = 2 * warp + (lane >> 4);
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
    // the activations: 8 lanes a block, 4 values a lane (whole warps run every round)
    for (int i0 = warp * 32; i0 < TN * nb * 8; i0 += kVecWarps * 32) {
        const int i = i0 + lane, q = i & 7, tb = i >> 3, t = TN > 1 && tb >= nb ? 1 : 0, b = tb - t * nb;
        uint32_t code;
        float dd;
        int sum;
        code_word(p, t, b, q, tb < TN * nb, code, dd, sum);
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        if (tb >= TN * nb) continue;
        ((uint32_t *)(q < 4 ? x0 : x1))[tb * 4 + (q & 3)] = code;
        if (q == 0) xs[tb] = BlockScale{dd, sum};
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
                if (b < nb)
#pragma unroll
                    for (int t = 0; t < TN; ++t)
                        acc[t] = w[i].term(q4_dot_raw(w[i].c, x0[t * nb + b], x1[t * nb + b]), xs[t * nb + b], acc[t]);
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
            if (row < p.rows && t < p.n_tokens) p.y[(size_t)t * p.rows + row] = v;
        }
    }
}

// ---- launch ---------------------------------------------------------------------
template <typename K>
int launch_pdl(K kernel, dim3 grid, unsigned block, size_t smem, const LinearParams &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, kernel, p);
}

// The kernel may use up to kLinearSmem bytes on the current device (asked once).
template <typename K>
int allow_smem(K kernel, bool (&done)[64]) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && done[dev]) return 0;
    const int rc = (int)cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinearSmem);
    if (!rc && dev >= 0 && dev < 64) done[dev] = true;
    return rc;
}

template <int FMT, int MT, int NT, int WC, bool RES>
int launch_tile(LinearParams p, int wr, int n_sm, cudaStream_t st) {
    static bool done[64];
    auto kernel = linear_kernel<FMT, MT, NT, WC, RES>;
    int rc = allow_smem(kernel, done);
    if (rc) return rc;
    const int nb = p.cols / kBlock, ng = (nb + kKB - 1) / kKB;
    const size_t stage = (size_t)wr * MT * group_bytes(FMT, kKB) + (RES ? 0 : (size_t)NT * WC * kKB * act_bytes(FMT));
    const size_t fixed = (RES ? (size_t)NT * WC * nb * act_bytes(FMT) : 0) +
                         (kNW / (WC * wr) > 1 ? (size_t)kNW / 2 * MT * NT * 512 : 0) + 512;
    const int tiles = ((p.rows + 16 * MT * wr - 1) / (16 * MT * wr)) * ((p.n_tokens + 8 * NT * WC - 1) / (8 * NT * WC));
    const int grid = std::min(tiles, n_sm), need = std::max(2, ng * ((tiles + grid - 1) / grid));
    p.wr = wr;
    p.stages = (int)std::min<size_t>({(kLinearSmem - fixed) / stage, (size_t)need, (size_t)16});
    if (p.stages < 2) return (int)cudaErrorInvalidValue;
    // stages split as many ways as the ring holds whole turns of
    p.ws_n = kNW / (WC * wr);
    while (p.ws_n > p.stages) p.ws_n /= 2;
    p.stages = p.stages / p.ws_n * p.ws_n;
    rc = launch_pdl(linear_prepare_kernel, dim3((unsigned)((p.n_tokens + 7) / 8), (unsigned)((nb + 3) / 4)), 256, 0, p,
                    st);
    return rc ? rc : launch_pdl(kernel, dim3((unsigned)grid), kNW * 32, p.stages * stage + fixed, p, st);
}

// Time of a row split, in rows: rounds of tiles over the SMs times a tile's
// rows and 16 rows' worth for each tile.
long split_cost(const LinearParams &p, int h, int nt, int n_sm) {
    const long tiles = (p.rows + h - 1L) / h * ((p.n_tokens + 8 * nt - 1) / (8 * nt));
    return (tiles + n_sm - 1) / n_sm * (h + 16);
}

template <int FMT, int NT>
int launch_small(const LinearParams &p, int n_sm, cudaStream_t st) {
    int best = 256;
    for (int h = 128; h >= 32; h /= 2)
        if (split_cost(p, h, NT, n_sm) < split_cost(p, best, NT, n_sm)) best = h;
    if (p.n_tokens <= 8 * NT && (size_t)NT * (p.cols / kBlock) * act_bytes(FMT) <= kLinearResident) {
        if (best == 32) return launch_tile<FMT, 1, NT, 1, true>(p, 2, n_sm, st);
        return launch_tile<FMT, 2, NT, 1, true>(p, best / 32, n_sm, st);
    }
    if (best == 32) return launch_tile<FMT, 1, NT, 1, false>(p, 2, n_sm, st);
    return launch_tile<FMT, 2, NT, 1, false>(p, best / 32, n_sm, st);
}

template <int FMT, int TN>
int launch_vec(const LinearParams &p, int n_sm, cudaStream_t st) {
    static bool done[64];
    const int rc = allow_smem(linear_vec_kernel<FMT, TN>, done);
    if (rc) return rc;
    const size_t smem = (size_t)TN * (p.cols / kBlock) * (32 + sizeof(BlockScale));
    const int fit = (int)std::max<size_t>(1, std::min<size_t>(4, kLinearSmem / (smem + 2048)));
    return launch_pdl(linear_vec_kernel<FMT, TN>, dim3((unsigned)std::min((p.rows + 15) / 16, n_sm * fit)),
                      kVecWarps * 32, smem, p, st);
}

template <int FMT>
int launch_fmt(const LinearParams &p, int n_sm, cudaStream_t st) {
    if (p.n_tokens == 1) return launch_vec<FMT, 1>(p, n_sm, st);
    if (p.n_tokens == 2 && 2 * (p.cols / kBlock) * 40 <= kLinearSmem) return launch_vec<FMT, 2>(p, n_sm, st);
    const int nt = (p.n_tokens + 7) / 8;
    if (nt == 1) return launch_small<FMT, 1>(p, n_sm, st);
    if (nt == 2) return launch_small<FMT, 2>(p, n_sm, st);
    if (nt <= 4) return launch_small<FMT, 4>(p, n_sm, st);
    // 256 rows x 64 tokens where that fills three quarters of the SMs
    if ((long)((p.rows + 255) / 256) * ((nt + 7) / 8) * 4 >= 3L * n_sm)
        return launch_tile<FMT, 2, 4, 2, false>(p, 8, n_sm, st);
    if (nt == 5) return launch_small<FMT, 5>(p, n_sm, st);
    if (nt == 6) return launch_small<FMT, 6>(p, n_sm, st);
    return launch_small<FMT, 8>(p, n_sm, st);
}

}  // namespace

size_t linear_weight_bytes(int fmt, int rows, int cols) {
    return (size_t)((rows + 15) / 16) * tile_bytes(fmt, cols / kBlock);
}
size_t linear_ws_bytes(int max_tokens, int cols) {
    return (size_t)((max_tokens + 7) / 8) * (cols / kBlock) * act_bytes(kFmtQ4K);
}

int launch_linear_repack(const uint8_t *src, uint8_t *dst, int fmt, int rows, int cols, int n_sm, cudaStream_t st) {
    const size_t n = (size_t)((rows + 15) / 16) * 16 * (cols / kBlock);
    const unsigned g = (unsigned)std::min<size_t>((n + 255) / 256, (size_t)n_sm * 8);
    linear_repack_kernel<<<g, 256, 0, st>>>(src, dst, fmt, rows, cols / kBlock);
    return (int)cudaGetLastError();
}

int launch_linear(const LinearParams &p, int n_sm, cudaStream_t st) {
    return p.fmt == kFmtQ4K ? launch_fmt<kFmtQ4K>(p, n_sm, st) : launch_fmt<kFmtQ4>(p, n_sm, st);
}

}  // namespace moe
