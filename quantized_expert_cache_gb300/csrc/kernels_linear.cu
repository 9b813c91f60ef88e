// y = W x of a dense layer with 4-bit weights and group scales, from one token
// to prompt chunks, on the library's int8 blocks.
//
//   y[t][r] = sum_b term(W block (r, b), x block (t, b)), block dots exact,
//   Q4_0: d_w d_a sum_i (q_w,i - 8) q_a,i
//   Q4_K: d sc_j d_a sum_i q_w,i q_a,i - dmin m_j d_a sum_i q_a,i
//
// Block dots on the tensor cores, exactly: a nibble under the binary16 exponent
// 0x64 is 1024 + q, an activation code is a binary16 integer, and the two
// m16n8k16 products of a block start from -1032 (Q4_K: -1024) times the code
// sum, so that they end at the block's dot; every partial sum is an integer
// below 2^23, which fp32 holds.  The sums stay in registers and their scaling
// costs two packed fp32 operations for two sums.  That is why this runs on
// mma.sync (594 TFLOP/s of f16 measured; s8 151, dp4a 149, e4m3 lowered to
// f16): tcgen05 leaves its sums in TMEM, where reading every block's sums back
// bounds the experts' GEMM at 0.07 of the peak, and folding the scales into two
// binary16 parts of each operand (three tcgen05 products a step, weights
// through TMEM) measured 63 us for 4096 x 4096 at 512 tokens, with larger
// errors.
//
// Weight layout (made at registration): per 16 rows, per group of up to 8
// blocks: the codes in the instruction's operand order, [block][lane] x 8
// bytes (lane 4g + t: elements 8t.. of row g, of row g + 8, nibble p of a word
// element 2p, nibble p + 4 element 2p + 1), then the scales:
// Q4_0 [block][g] x (binary16 d of rows g, g + 8); Q4_K [block][g] x bytes
// (sc, m of row g; of row g + 8), then [g] x (d, dmin of row g; of row g + 8).
// 18 (Q4_K 18.5) bytes to 32 weights, and any run of groups of 16 rows is one
// contiguous copy.
//
// Activation layout: per 8 tokens, per block, 576 bytes: [lane] x 16 (lane
// 4c + t: the codes 8t.. of token c in binary16), then [t] x 16: d_a of tokens
// 2t, 2t + 1, and what their products start from.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace moe {
namespace {

using namespace gemm;

constexpr int kKB = 8;            // blocks of a group: a pipeline stage
constexpr int kARec = 16 * 18;    // bytes of 16 rows of a Q4_0 block
constexpr int kBRec = 576;        // bytes of 8 tokens of a block

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
        // element e: byte e % 16, low nibble for e < 16
        const auto code = [&](int e) { return (w[(e & 15) >> 2] >> (8 * (e & 3) + (e >> 4) * 4)) & 15u; };
        for (int t = 0; t < 4; ++t) {
            uint32_t v = 0;
            for (int k = 0; k < 4; ++k) v |= code(8 * t + 2 * k) << (4 * k) | code(8 * t + 2 * k + 1) << (4 * k + 16);
            *(uint32_t *)(grp + bi * 256 + (4 * g + t) * 8 + up * 4) = v;
        }
    }
}

// ---- activations --------------------------------------------------------------
// Word w (elements 4w..4w+3) of token t's block b: the code word, the scale
// and, over the block's 8 lanes, the code sum.  All lanes of a warp call.
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
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
}

// ... into the 576-byte record of its block, token column c of 8.
__device__ __forceinline__ void put_word(uint8_t *rec, int c, int w, uint32_t code, float dd, int sum, int fmt) {
    // codes + 128 under the binary16 exponent 0x64: 1152 + q
    const uint32_t u = code ^ 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t h[2] = {__byte_perm(u, 0x64646464u, 0x4140), __byte_perm(u, 0x64646464u, 0x4342)};
#pragma unroll
    for (int i = 0; i < 2; ++i) *(__half2 *)&h[i] = __hsub2(*(__half2 *)&h[i], off);
    *((uint2 *)(rec + (4 * c + (w >> 1)) * 16) + (w & 1)) = make_uint2(h[0], h[1]);
    if (w == 0) {
        float *s = (float *)(rec + 512 + (c >> 1) * 16) + (c & 1);
        s[0] = dd;
        s[2] = (fmt == kFmtQ4K ? -1024.0f : -1032.0f) * (float)sum;
    }
}

// Records of 8 tokens (blockIdx.x) x 4 blocks (blockIdx.y) to the workspace;
// tokens past the last are zeros.
__global__ void __launch_bounds__(256) linear_prepare_kernel(LinearParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ __align__(16) uint8_t rec[4 * kBRec];
    const int nb = p.cols / kBlock, w = threadIdx.x & 7, c = (threadIdx.x >> 3) & 7, bi = threadIdx.x >> 6;
    const int b = blockIdx.y * 4 + bi, t = blockIdx.x * 8 + c, n = min(4, nb - (int)blockIdx.y * 4);
    uint32_t code;
    float dd;
    int sum;
    code_word(p, t, b, w, t < p.n_tokens && b < nb, code, dd, sum);
    put_word(rec + bi * kBRec, c, w, code, dd, sum, p.fmt);
    __syncthreads();
    uint4 *out = (uint4 *)(p.ws + ((size_t)blockIdx.x * nb + blockIdx.y * 4) * kBRec);
    for (int i = threadIdx.x; i < n * (kBRec / 16); i += 256) out[i] = ((const uint4 *)rec)[i];
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
    F2 s[2], m[2];  // scale of each row, twice; Q4_K: its min / 1024, twice
    __device__ __forceinline__ void load(const uint8_t *grp, int n, int b, int lane) {
        const uint2 c = *(const uint2 *)(grp + b * 256 + lane * 8);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[2 * k] = ((c.x >> (4 * k)) & 0x000F000Fu) | 0x64006400u;
            a[2 * k + 1] = ((c.y >> (4 * k)) & 0x000F000Fu) | 0x64006400u;
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
            const float s0 = d0.x * (v0.x - 1024.0f), m0 = d0.y * (v0.y - 1024.0f) * 0x1p-10f;
            const float s1 = d1.x * (v1.x - 1024.0f), m1 = d1.y * (v1.y - 1024.0f) * 0x1p-10f;
            s[0] = f2(s0, s0);
            m[0] = f2(m0, m0);
            s[1] = f2(s1, s1);
            m[1] = f2(m1, m1);
        }
    }
};

// where the activations' records come from
constexpr int kRing = 0;      // workspace, a stage with the weights' stages
constexpr int kResident = 1;  // workspace, all blocks in shared memory
constexpr int kStaged = 2;    // x or q and d, made in shared memory

// CTA tile: wr x MT x 16 rows, WC x NT x 8 tokens; its NW consumer warps split
// the rows wr ways, the tokens WC ways and the blocks of a stage wk ways.  CTAs
// walk the tiles (token tiles innermost: they share the weights in L2).  The
// producer warp copies group after group into a ring of stages.
template <int FMT, int MT, int NT, int WC, int NW, int MODE>
__global__ void __launch_bounds__((NW + 1) * 32, 1) linear_kernel(const __grid_constant__ LinearParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int wr_n = p.wr, wk_n = NW / (WC * wr_n), nb = p.cols / kBlock, ng = (nb + kKB - 1) / kKB;
    constexpr int NTC = NT * WC, GB = group_bytes(FMT, kKB), BST = kKB * kBRec;
    const int a_stage = wr_n * MT * GB, stage = a_stage + (MODE == kRing ? NTC * BST : 0);
    uint8_t *resident = smem + p.stages * stage;
    float4 *red = (float4 *)(resident + (MODE == kRing ? 0 : (size_t)NTC * nb * kBRec));
    uint64_t *bars = (uint64_t *)(red + (wk_n > 1 ? NW * MT * NT * 32 : 0));
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * p.stages, bfull = empty0 + 8 * p.stages;
    volatile int *abort_flag = (volatile int *)(bars + 2 * p.stages + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, NW);
        }
        mbar_init(bfull, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    const int rt_n = (p.rows + 15) / 16, tile_rt = wr_n * MT, ntt = (p.n_tokens + 8 * NTC - 1) / (8 * NTC);
    const int total = ((rt_n + tile_rt - 1) / tile_rt) * ntt, nt_n = (p.n_tokens + 7) / 8;
    const size_t rt_bytes = tile_bytes(FMT, nb);

    if (warp == NW) {
        // producer: lanes 0..tile_rt-1 copy a row tile's group, and (kRing)
        // lanes 0..NTC-1 the tokens' records of the group
        bool waited = MODE != kRing;  // the weights are the context's own; the records the preceding kernel's
        if (MODE == kResident) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            asm volatile("griddepcontrol.launch_dependents;");
            const int n = min(NTC, nt_n);
            if (lane == 0) mbar_arrive_tx(bfull, (uint32_t)(n * nb * kBRec));
            __syncwarp();
            if (lane < n)
                bulk_load(smem_u32(resident + (size_t)lane * nb * kBRec), p.ws + (size_t)lane * nb * kBRec,
                          (uint32_t)(nb * kBRec), bfull);
        }
        int it = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x) {
            const int rt0 = t / ntt * tile_rt, n_rt = min(tile_rt, rt_n - rt0);
            const int nt0 = t % ntt * NTC, n_nt = MODE == kRing ? min(NTC, nt_n - nt0) : 0;
            for (int g = 0; g < ng; ++g, ++it) {
                const int slot = it % p.stages, n = min(kKB, nb - g * kKB);
                const uint32_t full = full0 + 8 * slot, dst = smem_u32(smem + slot * stage);
                bool ok = true;
                if (lane == 0) {
                    ok = mbar_wait(empty0 + 8 * slot, ((uint32_t)(it / p.stages) & 1u) ^ 1u, abort_flag, p.error, 2);
                    if (ok)
                        mbar_arrive_tx(full, (uint32_t)(n_rt * group_bytes(FMT, n) + n_nt * n * kBRec));
                }
                if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) goto done;
                for (int i = lane; i < n_rt; i += 32)
                    bulk_load(dst + i * GB, p.w + (size_t)(rt0 + i) * rt_bytes + (size_t)g * GB, group_bytes(FMT, n),
                              full);
                if (MODE == kRing) {
                    if (!waited) {
                        asm volatile("griddepcontrol.wait;" ::: "memory");
                        asm volatile("griddepcontrol.launch_dependents;");
                        waited = true;
                    }
                    if (lane < n_nt)
                        bulk_load(dst + a_stage + lane * BST, p.ws + ((size_t)(nt0 + lane) * nb + g * kKB) * kBRec,
                                  (uint32_t)(n * kBRec), full);
                }
            }
        }
    done:;
    } else {
        const int wc = warp % WC, wr = warp / WC % wr_n, wk = warp / (WC * wr_n);
        if (MODE == kStaged) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            asm volatile("griddepcontrol.launch_dependents;");
            for (int i0 = warp * 32; i0 < 8 * NTC * nb * 8; i0 += NW * 32) {
                const int i = i0 + lane, w = i & 7, b = (i >> 3) % nb, t = (i >> 3) / nb;
                uint32_t code;
                float dd;
                int sum;
                code_word(p, t, b, w, t < p.n_tokens, code, dd, sum);
                if (t < 8 * NTC) put_word(resident + ((size_t)(t >> 3) * nb + b) * kBRec, t & 7, w, code, dd, sum, FMT);
            }
            asm volatile("bar.sync 1, %0;" ::"n"(NW * 32) : "memory");
        } else if (MODE == kResident) {
            mbar_wait(bfull, 0, abort_flag, p.error, 4);
        }
        int it = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x) {
            F2 acc[MT][NT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = f2(0.0f, 0.0f);
            for (int g = 0; g < ng; ++g, ++it) {
                const int slot = it % p.stages, n = min(kKB, nb - g * kKB);
                // a wait that expires leaves garbage and an error bit; the warp goes on, so that
                // the others' barriers complete
                mbar_wait(full0 + 8 * slot, (uint32_t)(it / p.stages) & 1u, abort_flag, p.error, 4);
                const uint8_t *ga = smem + slot * stage + wr * MT * GB;
                const uint8_t *gb = MODE == kRing ? smem + slot * stage + a_stage + wc * NT * BST
                                                  : resident + (size_t)g * kKB * kBRec;
                const size_t b_tile = MODE == kRing ? BST : (size_t)nb * kBRec;
#pragma unroll 2
                for (int b = wk; b < n; b += wk_n) {
                    WFrag<FMT> wf[MT];
#pragma unroll
                    for (int m = 0; m < MT; ++m) wf[m].load(ga + m * GB, n, b, lane);
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        const uint8_t *rec = gb + c * b_tile + b * kBRec;
                        const uint4 x = *(const uint4 *)(rec + lane * 16);
                        const float4 sc = *(const float4 *)(rec + 512 + (lane & 3) * 16);
                        const F2 da = f2(sc.x, sc.y);
                        float d[MT][4];
#pragma unroll
                        for (int m = 0; m < MT; ++m) mma_f16_sync(d[m], wf[m].a, x.x, x.y, sc.z, sc.w, sc.z, sc.w);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
                            mma_f16_sync(d[m], wf[m].a + 4, x.z, x.w, d[m][0], d[m][1], d[m][2], d[m][3]);
                        // Q4_K: -1024 d_a sum q_a times min / 1024
                        const F2 e = FMT == kFmtQ4K ? mul2(da, f2(sc.z, sc.w)) : da;
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
            }
            // lane 4g + q: rows g, g + 8 of a 16-row tile, tokens 2q, 2q + 1
            const int row0 = (t / ntt * tile_rt + wr * MT) * 16 + (lane >> 2);
            const int tok0 = (t % ntt * NTC + wc * NT) * 8 + (lane & 3) * 2;
            auto store = [&](int m, int c, const float4 &v) {
                const int row = row0 + m * 16, tok = tok0 + c * 8;
                float *y = p.y + (size_t)tok * p.rows + row;
                if (tok < p.n_tokens) {
                    if (row < p.rows) y[0] = v.x;
                    if (row + 8 < p.rows) y[8] = v.z;
                }
                if (tok + 1 < p.n_tokens) {
                    if (row < p.rows) y[p.rows] = v.y;
                    if (row + 8 < p.rows) y[(size_t)p.rows + 8] = v.w;
                }
            };
            if (wk_n == 1) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        const float2 u = un2(acc[m][c][0]), v = un2(acc[m][c][1]);
                        store(m, c, make_float4(u.x, u.y, v.x, v.y));
                    }
            } else {
                // the warps of one row and token share add up in block order
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        const float2 u = un2(acc[m][c][0]), v = un2(acc[m][c][1]);
                        red[(warp * MT * NT + m * NT + c) * 32 + lane] = make_float4(u.x, u.y, v.x, v.y);
                    }
                asm volatile("bar.sync 1, %0;" ::"n"(NW * 32) : "memory");
                for (int i = wk; i < MT * NT; i += wk_n) {
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int k = 0; k < wk_n; ++k) {
                        const float4 u = red[(((k * wr_n + wr) * WC + wc) * MT * NT + i) * 32 + lane];
                        v.x += u.x;
                        v.y += u.y;
                        v.z += u.z;
                        v.w += u.w;
                    }
                    store(i / NT, i % NT, v);
                }
                asm volatile("bar.sync 1, %0;" ::"n"(NW * 32) : "memory");
            }
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

// ---- launch ---------------------------------------------------------------------
template <int FMT, int MT, int NT, int WC, int NW, int MODE>
int launch_tile(LinearParams p, int wr, int n_sm, cudaStream_t st) {
    auto kernel = linear_kernel<FMT, MT, NT, WC, NW, MODE>;
    const int nb = p.cols / kBlock, ng = (nb + kKB - 1) / kKB;
    const size_t stage = (size_t)wr * MT * group_bytes(FMT, kKB) + (MODE == kRing ? (size_t)NT * WC * kKB * kBRec : 0);
    const size_t fixed = (MODE == kRing ? 0 : (size_t)NT * WC * nb * kBRec) +
                         (NW / (WC * wr) > 1 ? (size_t)NW * MT * NT * 512 : 0) + 512;
    const int tiles = ((p.rows + 16 * MT * wr - 1) / (16 * MT * wr)) * ((p.n_tokens + 8 * NT * WC - 1) / (8 * NT * WC));
    const int grid = std::min(tiles, n_sm), need = ng * ((tiles + grid - 1) / grid);
    p.wr = wr;
    p.stages = (int)std::min<size_t>({(kLinearSmem - fixed) / stage, (size_t)need, (size_t)16});
    if (p.stages < 1) return (int)cudaErrorInvalidValue;
    static bool configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinearSmem);
        if (e != cudaSuccess) return (int)e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((NW + 1) * 32);
    cfg.dynamicSmemBytes = p.stages * stage + fixed;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, kernel, p);
}

// The row split of the least time: rounds of tiles over the SMs times a tile's
// rows, a fixed cost of 16 rows' worth for each tile; the tallest of equals.
int pick_wr(const LinearParams &p, int mt, int nt, int n_sm) {
    int best = 8;
    long cost = -1;
    for (int wr = 8; wr >= 1; wr /= 2) {
        const long h = 16L * mt * wr, tiles = (p.rows + h - 1) / h * ((p.n_tokens + 8 * nt - 1) / (8 * nt));
        const long c = (tiles + n_sm - 1) / n_sm * (h + 16);
        if (cost < 0 || c < cost) {
            cost = c;
            best = wr;
        }
    }
    return best;
}

int launch_prepare(const LinearParams &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((p.n_tokens + 7) / 8), (unsigned)((p.cols / kBlock + 3) / 4));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, linear_prepare_kernel, p);
}

template <int FMT, int MT, int NT, int NW>
int launch_small(const LinearParams &p, int n_sm, cudaStream_t st) {
    const int wr = pick_wr(p, MT, NT, n_sm);
    const size_t records = (size_t)NT * (p.cols / kBlock) * kBRec;
    if (p.n_tokens <= 8 * NT && records <= kLinearResident) {
        if (p.n_tokens == 1) return launch_tile<FMT, MT, NT, 1, NW, kStaged>(p, wr, n_sm, st);
        const int rc = launch_prepare(p, st);
        return rc ? rc : launch_tile<FMT, MT, NT, 1, NW, kResident>(p, wr, n_sm, st);
    }
    const int rc = launch_prepare(p, st);
    return rc ? rc : launch_tile<FMT, MT, NT, 1, NW, kRing>(p, wr, n_sm, st);
}

template <int FMT>
int launch_fmt(const LinearParams &p, int n_sm, cudaStream_t st) {
    const int nt = (p.n_tokens + 7) / 8;
    if (nt == 1) {
        if (p.rows <= 16 * n_sm) return launch_small<FMT, 1, 1, 16>(p, n_sm, st);
        return launch_small<FMT, 2, 1, 16>(p, n_sm, st);
    }
    if (nt == 2) return launch_small<FMT, 2, 2, 16>(p, n_sm, st);
    if (nt <= 4) return launch_small<FMT, 2, 4, 8>(p, n_sm, st);
    // 256 rows x 64 tokens where that fills the SMs
    if ((long)((p.rows + 255) / 256) * ((nt + 7) / 8) * 4 >= 3L * n_sm) {
        const int rc = launch_prepare(p, st);
        return rc ? rc : launch_tile<FMT, 4, 4, 2, 8, kRing>(p, 4, n_sm, st);
    }
    if (nt == 5) return launch_small<FMT, 2, 5, 8>(p, n_sm, st);
    if (nt == 6) return launch_small<FMT, 2, 6, 8>(p, n_sm, st);
    return launch_small<FMT, 2, 8, 8>(p, n_sm, st);
}

}  // namespace

size_t linear_weight_bytes(int fmt, int rows, int cols) {
    return (size_t)((rows + 15) / 16) * tile_bytes(fmt, cols / kBlock);
}
size_t linear_ws_bytes(int max_tokens, int cols) {
    return (size_t)((max_tokens + 7) / 8) * (cols / kBlock) * kBRec;
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
