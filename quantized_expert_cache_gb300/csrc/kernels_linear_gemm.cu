// y = W x of a dense 4-bit layer for batches: the 5th-generation tensor cores
// (tcgen05, accumulators in TMEM), with the block scales folded into the
// operands instead of applied to block sums.
//
// Arithmetic.  A Q4_0 weight d (q - 8) has at most 15 significant bits and an
// activation d_a q_a at most 18, so neither fits one binary16; two do:
//   w = w_h + w_l,  x 2^-e = x_h + x_l   (each part the binary16 rounding of what
// is left, w_l below 2^-11 of w; exact, but for parts below binary16's smallest
// normal number, which are rounded to 2^-25: 2^e brings 127 times the token's
// largest scale to [2^13.9, 2^15), so that is 2^-38 of it) and
//   y = 2^e (sum w_h x_h  +  sum (w_l x_h + w_h x_l)),
// dropping w_l x_l (below 2^-22 of the product; with what the accumulation loses
// 6e-7 of the result measured at 4096 columns, 1.1e-6 for an fp32 library
// product).  Three MMAs a K step replace a scaled epilogue for every 32 columns:
// the exact-block-sum GEMM of the experts has to read every block's sums back
// from TMEM and is bound by that; exact block sums on mma.sync, scaled in
// registers, measured 88 us for 4096 x 4096 at 512 tokens (its f16 rate is a
// third of tcgen05's).  Q4_K weights are formed in binary32 (d sc q - dmin m),
// scaled by a power of two so that the largest of their row is below 2^15, and
// split the same way: to 2^-22 of themselves or 2^-38 of the row's largest.  (One
// power of two for the layer left rows far below its largest block to
// binary16's subnormals: 1e-3 off beside a block of d = 65504.)
//
// The tensor core's fp32 accumulation truncates, a bias of about 2^-24 a step
// on a growing sum; so the large products are accumulated for 512 columns
// only, then added in registers, rounded to nearest.  The cross
// products are 2^-11 of them and keep one accumulator for the whole tile.
//
// The weight halves go from the converters' registers to TMEM (tcgen05.st) and
// the MMA takes its A operand there: with A in shared memory an MMA reads 4 KB
// more (46 cycles at N = 32 against 26, 52 at N = 64 against 36; 64 at N = 128).
//
// Bound.  4096 x 4096 at 512 tokens: 48.8 us (51.5 GFLOP of MMAs, both
// kernels' time: 0.54 of the measured bf16 rate; Q4_K 56.0), the tensor pipe
// active 57% of the GEMM's time; 2880 x 2880 at 12288 tokens 559 us.  By count, not
// measured: operand reads, the tokens' copies and the weights' move about 90 KB
// through shared memory in a stage's 768 tensor cycles, near 128 bytes a cycle.
// Tiles of up to 64 tokens: the conversions, on four warps a scheduler: 65536 x
// 2048 at 5, 16 and 64 tokens 45, 47 and 54 us (Q4_K at 16 tokens 69), 2880 x 2880
// at 8 tokens 8.7 (latency of two launches, one round of stages and the join), Q4_K
// 8192 x 2048 at 33 tokens 15.7.
#include <cuda.h>
#include <cooperative_groups.h>

#include <algorithm>

#include "kernels.h"
#include "linear.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

using namespace gemm;

constexpr int kBM = 128;         // tile rows
constexpr int kConv = 16, kEpi = 8;  // converter and epilogue warps
constexpr int kWTma = 0, kWMma = 1;
constexpr int kBox = 32;         // token rows of one TMA box
constexpr int kAhead = 3;        // groups of weights (256 columns) in flight

// BN tokens a tile: 32, 64 or 128.  128 halves the conversions a token costs and
// leaves TMEM room for one buffer of the large products' sums only; its 64 sums
// an epilogue thread take registers from the other warps.
template <int FMT, int BN>
struct LCfg {
    static constexpr bool WIDE = BN == 128;
    static constexpr int BK = WIDE ? 64 : 128;           // columns of a stage
    static constexpr int BPS = BK / 32, SPG = 256 / BK;  // blocks of a stage, stages of a group
    static constexpr int CHUNK = 512 / BK;               // stages of a chunk
    static constexpr int WCONV = WIDE ? 4 : 2, WEPI = WCONV + kConv, THREADS = (WEPI + kEpi) * 32;
    static constexpr int ATOM = BN * 128, ATOMS = BK / 64;  // the tokens' 64 columns, a 128-byte swizzled row each
    static constexpr int SLOT = 2 * ATOMS * ATOM;        // high parts, low parts
    static constexpr int STAGES = 4;
    static constexpr int A_STAGES = WIDE ? 4 : 2;        // stages of weights in TMEM, BPS blocks of 32 columns each
    static constexpr int RED = BN * kBM * 4;             // a split tile's sums
    // weights on their way to the converters, [kAhead + 1] groups: of a thread's
    // two blocks the codes [2][thread] x 16, the scale words [2][thread] x 4 and
    // (Q4_K) d and dmin [thread] x 4
    static constexpr int CODES = 2 * kConv * 32 * 16, SCALES = 2 * kConv * 32 * 4;
    static constexpr int RAW_OFF = STAGES * SLOT > RED ? STAGES * SLOT : RED;
    static constexpr int RAW_BYTES = CODES + SCALES + (FMT == kFmtQ4K ? kConv * 32 * 4 : 0);
    static constexpr int BAR_OFF = RAW_OFF + (kAhead + 1) * RAW_BYTES;
    static constexpr int MISC_OFF = BAR_OFF + (2 * STAGES + 6) * 8;
    static constexpr int SMEM = MISC_OFF + 16;
    // TMEM columns: the large products' sums (two buffers if they fit), the
    // cross products', the weight blocks
    static constexpr int MAINS = WIDE ? 1 : 2;
    static constexpr int CROSS = MAINS * BN, A_COL = CROSS + BN, COLS = 512;
    static_assert(A_COL + 32 * BPS * A_STAGES <= COLS && A_STAGES <= STAGES, "TMEM");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// Register shares of the wide tile's warpgroups (28 warps of kRegs at launch):
// TMA and MMA, four of converters, two of the epilogue.
constexpr int kRegs = 72, kRegsLead = 40, kRegsConv = 64, kRegsEpi = 104;
static_assert(kRegsLead + 4 * kRegsConv + 2 * kRegsEpi <= 7 * kRegs, "registers");
template <int N, bool UP>
__device__ __forceinline__ void set_regs() {
    if (UP)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- activations: codes and scales -> the two halves -------------------------
// One CTA a token, four values a thread and round: ITEMS rounds in registers,
// or (ITEMS 0) any number, read twice.  FP: x, quantized here; else q and d.
template <bool FP, int ITEMS>
__global__ void __launch_bounds__(256) linear_split_kernel(LinearParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ unsigned part[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = p.cols, n4 = K / 4;
    const size_t t = blockIdx.x;
    struct Four {
        float v[4];  // FP: values; else codes
        float d;     // else: the block's scale
    };
    auto load = [&](int i) {
        Four f{};
        if (i >= n4) return f;
        if (FP) {
            *(float4 *)f.v = *((const float4 *)(p.x + t * K) + i);
        } else {
            const uint32_t w = *((const uint32_t *)(p.q + t * K) + i);
            f.d = __half2float(p.d[t * (n4 / 8) + i / 8]);
#pragma unroll
            for (int j = 0; j < 4; ++j) f.v[j] = (float)(int8_t)(w >> (8 * j));
        }
        return f;
    };
    // non-negative floats order like their bits (NaN above all)
    auto top4 = [](const Four &f) {
        return FP ? max(max(__float_as_uint(fabsf(f.v[0])), __float_as_uint(fabsf(f.v[1]))),
                        max(__float_as_uint(fabsf(f.v[2])), __float_as_uint(fabsf(f.v[3]))))
                  : __float_as_uint(fabsf(f.d));
    };
    Four held[ITEMS ? ITEMS : 1];
    unsigned m = 0;
    if (ITEMS) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) held[i] = load(threadIdx.x + 256 * i);
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) m = max(m, top4(held[i]));
    } else {
        for (int i = threadIdx.x; i < n4; i += 256) m = max(m, top4(load(i)));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) part[warp] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, part[lane & 7]);
    // the token's largest scale; the scales times 2^-e, which brings them below
    // 2^8 and the values (127 of them) below 2^15 (e = -7 for a token of zeros,
    // infinities or NaN)
    float top = __uint_as_float(m);
    if (FP) top = __half2float(__float2half_rn(top / 127.0f));
    const int e = (top > 0.0f && top <= 65504.0f ? (int)((__float_as_uint(top) >> 23) & 255u) - 127 : 0) - 7;
    const float up = __uint_as_float((unsigned)(127 + e) << 23), down = __uint_as_float((unsigned)(127 - e) << 23);
    if (threadIdx.x == 0) p.ws_scale[t] = up;
    // 8 lanes a block (whole warps run every round)
    auto emit = [&](int i, Four f) {
        if (FP) {
            unsigned a = top4(f);
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
            f.d = __half2float(__float2half_rn(__uint_as_float(a) / 127.0f));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f.v[j] = f.d != 0.0f ? fminf(fmaxf(rintf(f.v[j] / f.d), -127.0f), 127.0f) : 0.0f;
        }
        if (i >= n4) return;
        const float r = f.d * down;
        __half h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v = f.v[j] * r;
            h[j] = __float2half_rn(v);
            l[j] = __float2half_rn(v - __half2float(h[j]));
        }
        // the weights' order within a block: elements (0, 2) of word w & 3 at pair w >> 2, (1, 3) two pairs on
        const size_t o = (t * K + (size_t)(i & ~7) * 4) / 2 + (i & 3) * 4 + ((i >> 2) & 1);
        ((__half2 *)p.ws_hi)[o] = __halves2half2(h[0], h[2]);
        ((__half2 *)p.ws_hi)[o + 2] = __halves2half2(h[1], h[3]);
        ((__half2 *)p.ws_lo)[o] = __halves2half2(l[0], l[2]);
        ((__half2 *)p.ws_lo)[o + 2] = __halves2half2(l[1], l[3]);
    };
    if (ITEMS) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (warp * 32 + 256 * i < n4) emit(threadIdx.x + 256 * i, held[i]);
    } else {
        for (int i = threadIdx.x; i - lane < n4; i += 256) emit(i, load(i));
    }
}

template <bool FP>
int launch_split(const LinearParams &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.n_tokens);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.cols <= 1024) return (int)cudaLaunchKernelEx(&cfg, linear_split_kernel<FP, 1>, p);
    if (p.cols <= 2048) return (int)cudaLaunchKernelEx(&cfg, linear_split_kernel<FP, 2>, p);
    if (p.cols <= 4096) return (int)cudaLaunchKernelEx(&cfg, linear_split_kernel<FP, 4>, p);
    if (p.cols <= 8192) return (int)cudaLaunchKernelEx(&cfg, linear_split_kernel<FP, 8>, p);
    return (int)cudaLaunchKernelEx(&cfg, linear_split_kernel<FP, 0>, p);
}

// ---- weights: one block of 32 -> the two halves ------------------------------
template <int FMT>
struct WRaw {
    uint4 c;      // codes
    uint32_t s;   // scale bytes of rows g and g + 8
    uint32_t dm;  // Q4_K: this row's d and dmin
    int up;       // this row is the second of the two
    __device__ __forceinline__ void load(uint32_t codes, uint32_t scales, uint32_t mins) {
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(c.x), "=r"(c.y), "=r"(c.z), "=r"(c.w)
                     : "r"(codes)
                     : "memory");
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(s) : "r"(scales) : "memory");
        if (FMT == kFmtQ4K) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(dm) : "r"(mins) : "memory");
    }
};

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// Pair j of a code word (nibbles j and j + 4) as binary16 64 + q, exact.
__device__ __forceinline__ __half2 pair_q(uint32_t c, int j) {
    const uint32_t n = j == 0 ? c << 4 : c >> (4 * j - 4);
    return u2h((n & 0x00F000F0u) | 0x54005400u);
}

// The block's 32 weights: word i's four pairs in turn (elements 4i + (0, 2),
// 16 + 4i + (0, 2), 4i + (1, 3), 16 + 4i + (1, 3)), high parts h, low parts l.
// (Splitting Q4_0's scale into its upper 7 bits and the 4 below instead takes
// two operations a pair and not three, but makes w_l x_l 2^-20 of the product:
// 9e-7 of the result off instead of 6e-7, or a fourth product.)
__device__ __forceinline__ void convert(const WRaw<kFmtQ4> &w, float /*scale*/, uint32_t (&h)[16], uint32_t (&l)[16]) {
    const uint32_t c[4] = {w.c.x, w.c.y, w.c.z, w.c.w};
    const __half2 d = u2h(__byte_perm(w.s, 0, w.up ? 0x3232 : 0x1010)), m72 = __float2half2_rn(-72.0f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const __half2 q = __hadd2(pair_q(c[i >> 2], i & 3), m72);  // q - 8
        const __half2 v = __hmul2(q, d);
        h[i] = h2u(v);
        l[i] = h2u(__hfma2(q, d, __hneg2(v)));  // exact: 15 bits less the 11 above
    }
}

__device__ __forceinline__ void convert(const WRaw<kFmtQ4K> &w, float scale, uint32_t (&h)[16], uint32_t (&l)[16]) {
    const uint32_t c[4] = {w.c.x, w.c.y, w.c.z, w.c.w}, s = w.up ? w.s >> 16 : w.s;
    const float2 dm = __half22float2(u2h(w.dm));
    const float sc = dm.x * (float)(s & 255u) * scale, mn = dm.y * (float)((s >> 8) & 255u) * scale;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 q = __half22float2(pair_q(c[i >> 2], i & 3));
        const float v0 = fmaf(q.x - 64.0f, sc, -mn), v1 = fmaf(q.y - 64.0f, sc, -mn);
        const __half2 v = __floats2half2_rn(v0, v1);
        h[i] = h2u(v);
        l[i] = h2u(__floats2half2_rn(v0 - __low2float(v), v1 - __high2float(v)));
    }
}

// ---- the GEMM -----------------------------------------------------------------
// CTA tile: 128 weight rows (TMEM lanes) x BN tokens.  gridDim.x CTAs walk the
// tiles (token tiles innermost: they share the weight rows in L2).  A cluster
// of S > 1 CTAs (one tile each) splits K and joins its sums in shared memory,
// in rank order.
template <int FMT, int BN>
__global__ void __launch_bounds__((LCfg<FMT, BN>::THREADS), 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap tm_hi, const __grid_constant__ CUtensorMap tm_lo,
                       const __grid_constant__ LinearParams p) {
    using C = LCfg<FMT, BN>;
    constexpr int STAGES = C::STAGES;
    // (aligned by the declaration, so that addresses in it are constants: the
    // kernel has no other shared memory)
    extern __shared__ __align__(1024) uint8_t smem[];
    // full: a stage's tokens and weights are in place; done: its products are
    constexpr int AST = C::A_STAGES;
    const uint32_t full0 = smem_u32(smem + C::BAR_OFF), done0 = full0 + 8 * STAGES, accf0 = done0 + 8 * STAGES,
                   acce0 = accf0 + 16, crosse = acce0 + 16;
    volatile uint32_t *tmem_slot = (volatile uint32_t *)(smem + C::MISC_OFF);
    volatile int *abort_flag = (volatile int *)(smem + C::MISC_OFF + 4);
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1 + 4 * C::BPS);  // TMA expect-tx arrive + the blocks' converter warps
            mbar_init(done0 + 8 * s, 1);               // MMA commit
        }
        mbar_init(crosse, kEpi);
        for (int j = 0; j < 2; ++j) {
            mbar_init(accf0 + 8 * j, 1);
            mbar_init(acce0 + 8 * j, kEpi);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kWMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32((const void *)tmem_slot)),
                     "n"(C::COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // all 512 columns: the allocation starts at column 0, a constant
    constexpr uint32_t tmem = 0;
    const bool off = *tmem_slot != 0 || (smem_u32(smem) & 1023);  // never: then nothing is computed
    __syncthreads();
    if (off && threadIdx.x == 0) {
        *abort_flag = 1;
        atomicOr(p.error, 64);
    }

    const int nb = p.cols / kBlock, rt_n = (p.rows + 15) / 16, ng = (nb + kKB - 1) / kKB;
    // this CTA's K stages, whole groups of blocks (columns past the last are zeros)
    const int kt0 = C::SPG * (ng * rank / S), kt1 = C::SPG * (ng * (rank + 1) / S);
    const int ntt = (p.n_tokens + BN - 1) / BN, nrt = (p.rows + kBM - 1) / kBM;
    const int tile0 = blockIdx.x / S, total = off ? 0 : ntt * nrt, stride = gridDim.x / S;
    const auto columns = [&](int tt) { return min(BN, p.n_tokens - tt * BN); };

    if (C::WIDE && warp < C::WCONV) set_regs<kRegsLead, false>();
    if (warp == kWTma) {
        if (lane == 0) {
            // the split activations are the preceding kernel's
            asm volatile("griddepcontrol.wait;" ::: "memory");
            asm volatile("griddepcontrol.launch_dependents;");
            int it = 0;
            for (int t = tile0; t < total; t += stride) {
                const int tt = t % ntt, boxes = (columns(tt) + kBox - 1) / kBox;
                for (int kt = kt0; kt < kt1; ++kt, ++it) {
                    const int slot = it % STAGES;
                    if (!mbar_wait(done0 + 8 * slot, ((uint32_t)(it / STAGES) & 1u) ^ 1u, abort_flag, p.error, 2))
                        goto tma_done;
                    const uint32_t full = full0 + 8 * slot, b = smem_u32(smem + slot * C::SLOT);
                    mbar_arrive_tx(full, (uint32_t)(2 * C::ATOMS * boxes * kBox * 128));
                    for (int a = 0; a < C::ATOMS; ++a)  // 64 columns each; past the last they read zeros
                        for (int i = 0; i < boxes; ++i) {
                            const uint32_t dst = b + a * C::ATOM + i * kBox * 128;
                            tma_load_2d(dst, &tm_hi, kt * C::BK + a * 64, tt * BN + i * kBox, full);
                            tma_load_2d(dst + C::ATOMS * C::ATOM, &tm_lo, kt * C::BK + a * 64, tt * BN + i * kBox, full);
                        }
                }
            }
        tma_done:;
        }
    } else if (warp == kWMma) {
        {
            int it = 0, chunk = 0, n_tile = 0;
            for (int t = tile0; t < total; t += stride, ++n_tile) {
                const uint32_t idesc = idesc_f16(kBM, (columns(t % ntt) + 15) & ~15), cross = tmem + C::CROSS;
                // the cross sums of the tile before are read
                if (!mbar_wait_warp(crosse, ((uint32_t)n_tile & 1u) ^ 1u, abort_flag, p.error, 8)) goto mma_done;
                for (int kt = kt0; kt < kt1; ++kt, ++it) {
                    const int slot = it % STAGES, in_chunk = (kt - kt0) % C::CHUNK, buf = chunk % C::MAINS;
                    if (in_chunk == 0) {
                        if (!mbar_wait_warp(acce0 + 8 * buf, ((uint32_t)(chunk / C::MAINS) & 1u) ^ 1u, abort_flag, p.error, 8))
                            goto mma_done;
                    }
                    if (!mbar_wait_warp(full0 + 8 * slot, (uint32_t)(it / STAGES) & 1u, abort_flag, p.error, 4))
                        goto mma_done;
                    tc_fence_after();
                    const uint32_t st = smem_u32(smem + slot * C::SLOT), main = tmem + (uint32_t)(buf * BN);
                    const uint32_t a = tmem + (uint32_t)(C::A_COL + 32 * C::BPS * (it % AST));
                    const uint64_t bh = sdesc(st), bl = sdesc(st + C::ATOMS * C::ATOM);
#pragma unroll
                    for (int kk = 0; kk < C::BK / 16; ++kk) {
                        const uint32_t ah = a + 32 * (kk >> 1) + 8 * (kk & 1), al = ah + 16;
                        const uint64_t ko = (uint64_t)((kk >> 2) * C::ATOM + (kk & 3) * 32) >> 4;
                        mma_f16_ta(main, ah, bh + ko, idesc, in_chunk | kk ? 1u : 0u);
                        mma_f16_ta(cross, al, bh + ko, idesc, (kt - kt0) | kk ? 1u : 0u);
                        mma_f16_ta(cross, ah, bl + ko, idesc, 1u);
                    }
                    mma_commit_warp(done0 + 8 * slot);
                    if (in_chunk == C::CHUNK - 1 || kt == kt1 - 1) {
                        mma_commit_warp(accf0 + 8 * buf);
                        ++chunk;
                    }
                }
            }
        mma_done:;
        }
    } else if (warp < C::WCONV) {
        // (fills the first warpgroup)
    } else if (warp < C::WEPI) {
        // Converters: the four sets of four warps take blocks set and set + 4 of
        // every group.  A thread owns a row's block; the next kAhead groups' are on
        // their way to its own place in shared memory (asynchronous copies: a
        // register ring waited for its newest loads), and one is converted
        // before its place in TMEM (the row's lane) is waited for.
        if (C::WIDE) set_regs<kRegsConv, false>();
        const int set = (warp - C::WCONV) >> 2, quarter = warp & 3, row = quarter * 32 + lane, r = row & 15;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + C::A_COL + 32 * (set % C::BPS);
        const size_t rt_bytes = tile_bytes(FMT, nb);
        const int me = threadIdx.x - C::WCONV * 32;
        const uint32_t codes = smem_u32(smem + C::RAW_OFF) + me * 16,
                       scales = smem_u32(smem + C::RAW_OFF) + C::CODES + me * 4;
        int ft = tile0, fg = kt0 / C::SPG, fe = 0;  // fetch cursor
        const uint8_t *grp = nullptr;          // its group of its row tile
        bool live = false;                     // there is one
        auto aim = [&]() {
            const int rt = ft / ntt * (kBM / 16) + (row >> 4);
            live = ft < total && rt < rt_n;
            grp = live ? p.w + rt * rt_bytes + (size_t)(kt0 / C::SPG) * group_bytes(FMT, kKB) : p.w;
        };
        aim();
        auto fetch = [&]() {
            // blocks set and set + 4 of the group (its first n)
            const int n = min(kKB, nb - kKB * fg);
            const bool on0 = live && set < n, on1 = live && set + 4 < n;
            const uint8_t *c = grp + set * 256 + r * 16, *sc = grp + n * 256 + set * 32 + (r & 7) * 4;
            const uint32_t dc = codes + fe * C::RAW_BYTES, ds = scales + fe * C::RAW_BYTES;
            cp_async(dc, c, 16, on0);
            cp_async(dc + C::CODES / 2, c + 4 * 256, 16, on1);
            cp_async(ds, sc, 4, on0);
            cp_async(ds + C::SCALES / 2, sc + 4 * 32, 4, on1);
            if (FMT == kFmtQ4K) cp_async(ds + C::SCALES, grp + kKB * kARec + (r & 7) * 8 + (r >> 3) * 4, 4, live);
            cp_commit();
            fe = fe == kAhead ? 0 : fe + 1;
            if (live) grp += group_bytes(FMT, kKB);
            if (C::SPG * ++fg < kt1) return;
            fg = kt0 / C::SPG;
            ft += stride;
            aim();
        };
        for (int i = 0; i < kAhead; ++i) fetch();
        int ce = 0;
        bool ok = true;
        auto group = [&](int it0, float scale) {
            fetch();
            cp_wait<kAhead>();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                WRaw<FMT> raw;
                raw.load(codes + ce * C::RAW_BYTES + j * (C::CODES / 2), scales + ce * C::RAW_BYTES + j * (C::SCALES / 2),
                         scales + ce * C::RAW_BYTES + C::SCALES);
                raw.up = r >> 3;
                uint32_t h[16], l[16];
                convert(raw, scale, h, l);
                // block set + 4 j's stage; its place in TMEM was that of AST stages ago
                const int it = it0 + (set + 4 * j) / C::BPS, prev = it - AST;
                if (prev >= 0) {
                    const uint32_t bar = done0 + 8 * (prev % STAGES), parity = (uint32_t)(prev / STAGES) & 1u;
                    if (!__all_sync(0xffffffffu, mbar_test(bar, parity))) {
                        if (lane == 0) ok = mbar_wait(bar, parity, abort_flag, p.error, 16);
                        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                        if (!ok) break;
                    }
                }
                tc_fence_after();
                tmem_st16(lanes + 32 * C::BPS * (it % AST), h);
                tmem_st16(lanes + 32 * C::BPS * (it % AST) + 16, l);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                mbar_arrive_warp(full0 + 8 * (it % STAGES), lane);
            }
            ce = ce == kAhead ? 0 : ce + 1;
        };
        // Q4_K goes tile by tile, each with the power of two of this thread's row
        // (switched inside one loop over all groups, as Q4_0 has it, 65536 x 2048
        // at 16 tokens took 72 us instead of 69; Q4_0 by tiles 47.7 instead of 47.3)
        if constexpr (FMT == kFmtQ4K) {
            const float *row_scale = (const float *)(p.w + row_scale_offset(FMT, p.rows, nb)) + row;
            for (int t = tile0, it0 = 0; t < total && ok; t += stride) {
                const float scale = __ldg(row_scale + t / ntt * kBM);
                for (const int end = it0 + (kt1 - kt0); it0 < end && ok; it0 += C::SPG) group(it0, scale);
            }
        } else {
            const int n_it = tile0 < total ? ((total - 1 - tile0) / stride + 1) * (kt1 - kt0) : 0;
            for (int it0 = 0; it0 < n_it && ok; it0 += C::SPG) group(it0, 1.0f);
        }
        cp_wait<0>();
    } else {
        // Epilogue: TMEM lane quarter = warp % 4 (lane = weight row), one half
        // of the token columns.
        if (C::WIDE) set_regs<kRegsEpi, true>();
        constexpr int HC = BN / 2;
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int quarter = warp & 3, c0 = ((warp - C::WEPI) >> 2) * HC, r = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        int chunk = 0;
        for (int t = tile0; t < total; t += stride) {
            const int tt = t % ntt, nc = columns(tt) - c0;  // this warp's valid columns
            const int row = t / ntt * kBM + r;
            uint32_t rs = 0;  // Q4_K: the row's power of two
            if (FMT == kFmtQ4K) rs = __ldg((const uint32_t *)(p.w + row_scale_offset(FMT, p.rows, nb)) + row);
            float acc[HC];
#pragma unroll
            for (int i = 0; i < HC; ++i) acc[i] = 0.0f;
            // the columns' token scales (powers of two): lane i has columns i, i + 32
            float ts[(HC + 31) / 32];
#pragma unroll
            for (int i = 0; i < (HC + 31) / 32; ++i)
                ts[i] = lane + 32 * i < nc ? __ldcg(p.ws_scale + (size_t)tt * BN + c0 + lane + 32 * i) : 0.0f;
            auto add = [&](uint32_t col) {
#pragma unroll
                for (int i = 0; i < HC; i += 16) {
                    if (i >= nc) break;  // warp-uniform
                    uint32_t v[16];
                    tmem_ld16u(lanes + col + (uint32_t)(c0 + i), v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[i + j] += __uint_as_float(v[j]);
                }
            };
            for (int kt = kt0; kt < kt1; kt += C::CHUNK, ++chunk) {
                const int buf = chunk % C::MAINS;
                bool ok = true;
                if (lane == 0) ok = mbar_wait(accf0 + 8 * buf, (uint32_t)(chunk / C::MAINS) & 1u, abort_flag, p.error, 32);
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                if (!ok) goto epi_done;
                tc_fence_after();
                add((uint32_t)(buf * BN));
                tc_fence_before();
                __syncwarp();
                mbar_arrive_warp(acce0 + 8 * buf, lane);
                if (kt + C::CHUNK >= kt1) {
                    add(C::CROSS);
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_warp(crosse, lane);
                }
            }
            float *red = (float *)smem;  // a split tile: its sums [column][row], over the stages it is done with
#pragma unroll
            for (int i = 0; i < HC; ++i) {
                if (i >= nc) break;  // warp-uniform
                float v = acc[i] * __shfl_sync(0xffffffffu, ts[i / 32], i % 32);
                if (FMT == kFmtQ4K) v *= __uint_as_float((254u << 23) - rs);  // its inverse
                if (S > 1)
                    red[(c0 + i) * kBM + r] = v;
                else if (row < p.rows)
                    p.y[((size_t)tt * BN + c0 + i) * p.rows + row] = v;
            }
        }
    epi_done:;
    }

    __syncwarp();
    if (S > 1) {
        cluster.sync();
        if (warp >= C::WEPI && !*abort_flag) {
            const int tt = tile0 % ntt, nc = columns(tt), rt = tile0 / ntt;
            // four rows of a column a thread and round, all ranks' loads in flight
            const float4 *red = (const float4 *)smem;
            for (int i = threadIdx.x - C::WEPI * 32 + rank * kEpi * 32; i < nc * kBM / 4; i += S * kEpi * 32) {
                float4 v[8];
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (s < S) v[s] = *cluster.map_shared_rank(red + i, s);
                float sum[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
                for (int s = 1; s < 8; ++s)
                    if (s < S) {
                        sum[0] += v[s].x;
                        sum[1] += v[s].y;
                        sum[2] += v[s].z;
                        sum[3] += v[s].w;
                    }
                const int row = rt * kBM + i % (kBM / 4) * 4;
                float *y = p.y + ((size_t)tt * BN + i / (kBM / 4)) * p.rows + row;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (row + j < p.rows) y[j] = sum[j];
            }
        }
        __syncwarp();
        cluster.sync();  // no CTA leaves while its sums are read
    }
    // drain: after an abort, give the copies and MMAs this CTA issued a
    // bounded time (about 10 ms) to land, then free TMEM
    __syncthreads();
    if (*abort_flag) {
        const long long t0 = clock64();
        while (clock64() - t0 < 20000000ll) {
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*tmem_slot), "n"(C::COLS) : "memory");
}

// Tiles of BN tokens, and the K splits of one: as many as the SMs take, of at
// least a group of blocks.
int tiles_of(const LinearParams &p, int bn) {
    return (p.n_tokens + bn - 1) / bn * ((p.rows + kBM - 1) / kBM);
}
int groups_of(const LinearParams &p) { return (p.cols + kKB * kBlock - 1) / (kKB * kBlock); }
int splits_of(const LinearParams &p, int bn, int n_sm) {
    return std::max(1, std::min({8, n_sm / tiles_of(p, bn), groups_of(p)}));
}

template <int FMT, int BN>
int launch_tile(const LinearGemm &g, int n_sm, cudaStream_t st) {
    const LinearParams &p = g.p;
    auto kernel = linear_gemm_kernel<FMT, BN>;
    const int tiles = tiles_of(p, BN), S = splits_of(p, BN, n_sm);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(S > 1 ? tiles * S : std::min(tiles, n_sm)));
    cfg.blockDim = dim3(LCfg<FMT, BN>::THREADS);
    cfg.dynamicSmemBytes = LCfg<FMT, BN>::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)S, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return (int)cudaLaunchKernelEx(&cfg, kernel, g.tm_hi, g.tm_lo, p);
}

// The wide tile's kernel has the registers that its warpgroups share out.
template <int FMT>
bool wide_ok() {
    static int regs = -1;
    if (regs < 0) {
        cudaFuncAttributes a{};
        regs = cudaFuncGetAttributes(&a, linear_gemm_kernel<FMT, 128>) == cudaSuccess ? a.numRegs : 0;
    }
    return regs == kRegs;
}

// Clocks of the longest CTA: rounds of tiles x groups x a group's clocks (Q4_0:
// 2600 in a tile of 64 tokens, 4960 in one of 128, whose MMAs bound it; Q4_K:
// 3900, bound by the conversions, and 5000), and 3000 to join a split tile.
long clocks_of(const LinearParams &p, int bn, int n_sm, long group) {
    const int tiles = tiles_of(p, bn), S = splits_of(p, bn, n_sm);
    return (tiles * S + n_sm - 1L) / n_sm * ((groups_of(p) + S - 1) / S) * group + (S > 1 ? 3000 : 0);
}

// Up to 128 tokens one tile holds them all and weights are converted once; above,
// the shorter schedule.  us in tiles of 128 and of 64: Q4_0 80 x 1000 x 2048 (tokens,
// rows, columns) 12.9 and 15.4, 128 x 8192 x 8192 53.2 and 53.0, 128 x 2880 x 2880
// 18.8 and 17.0 (the rule's loss), 512 x 4096 x 4096 49.0 and 52.7, 512 x 16384 x
// 1024 57.2 and 51.9, 4096 x 2048 x 2048 102.9 and 97.3; Q4_K 100 x 1000 x 2048 14.5
// and 19.3, 128 x 8192 x 8192 59.7 and 75.5, 512 x 4096 x 4096 56.5 and 76.1.
template <int FMT>
int launch_fmt(const LinearGemm &g, int n_sm, cudaStream_t st) {
    if (g.p.n_tokens <= 32) return launch_tile<FMT, 32>(g, n_sm, st);
    const bool q4k = FMT == kFmtQ4K;
    const bool wide = g.p.n_tokens > 64 && wide_ok<FMT>() &&
                      (g.p.n_tokens <= 128 ||
                       clocks_of(g.p, 128, n_sm, q4k ? 5000 : 4960) <= clocks_of(g.p, 64, n_sm, q4k ? 3900 : 2600));
    return wide ? launch_tile<FMT, 128>(g, n_sm, st) : launch_tile<FMT, 64>(g, n_sm, st);
}

template <int FMT>
int configure_fmt() {
    cudaError_t e = cudaFuncSetAttribute(linear_gemm_kernel<FMT, 32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         LCfg<FMT, 32>::SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(linear_gemm_kernel<FMT, 64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 LCfg<FMT, 64>::SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(linear_gemm_kernel<FMT, 128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 LCfg<FMT, 128>::SMEM);
    return (int)e;
}

}  // namespace

int linear_gemm_box() { return kBox; }

int linear_gemm_configure() {
    const int rc = configure_fmt<kFmtQ4>();
    return rc ? rc : configure_fmt<kFmtQ4K>();
}

int launch_linear_gemm(const LinearGemm &g, int n_sm, cudaStream_t st) {
    const int rc = g.p.x ? launch_split<true>(g.p, st) : launch_split<false>(g.p, st);
    if (rc) return rc;
    return g.p.fmt == kFmtQ4K ? launch_fmt<kFmtQ4K>(g, n_sm, st) : launch_fmt<kFmtQ4>(g, n_sm, st);
}

}  // namespace moe
