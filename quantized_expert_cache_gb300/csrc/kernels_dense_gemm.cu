// The products of a 16-bit dense layer on the 5th-generation tensor cores: the layer
// itself, the gradient of its input and the gradient of its weights.
//
//   D[m][n] = sum_k A[m][k] B[n][k], m the contiguous direction of the result:
//   layer:    m = rows of W, n = tokens, k = columns:  A = W [m][k],  B = x [n][k]
//   input:    m = columns, n = tokens, k = rows of W:  A = W [k][m],  B = dz [n][k]
//   weights:  m = columns, n = rows of W, k = tokens:  A = x [k][m],  B = dz [k][n]
//
// An operand is read as it lies in memory: one whose k is contiguous as rows of 64 k
// (two blocks to a step), the other kind as rows of 64 m (or n), both in the 128-byte
// swizzle that the MMA's descriptors name; nothing is transposed.  A thread of the
// epilogue has one m and many n; blocks of them turn in shared memory, so that a lane
// stores four or eight neighbours of the result.
//
// The accumulators are drained every 512 of k (kChunk32) and added up in registers,
// rounded to nearest: the tensor core's own fp32 accumulation truncates, a bias of about
// 2^-24 a step on a growing sum.  Every 2048 (kChunk16) for 16-bit results, whose own
// rounding is 2^-12 and more, and for products of lower parts, which are small beside the
// last pair's: the drains' reads of TMEM hold the products up (8192^3 697 us at 512,
// 658 at 2048; 4096 x 8192 x 2048 115 and 103, in the forms of that time).  Two
// accumulators in turn hide most of it, and the epilogue of a tile behind the next one's
// products.
//
// Few tokens of fp32 rows: their parts are columns of B, four to a token (the fourth
// zero), and a token's four sums are added in the epilogue: the weights are read once
// (8 tokens on 65536 x 2048 47 us, 91 with a pass for each part).
//
// Where there are fewer tiles than SMs, a tile's steps are shared out over a cluster
// of CTAs and their sums joined through distributed shared memory, in order; or, in a
// weights' gradient, over tiles of their own whose sums are joined in the workspace.
//
// Bound.  8192^3 bf16 607 us, 4096^3 99, 4096 x 8192 x 2048 87, 4096 x 32000 x 2048 298 (the
// library's product 550, 79, 72 and 282; all with a cold cache); both gradients of 4096^3
// 171 (1610 TFLOP/s, 0.84 of the measured rate; tensor pipe active 77% of the time).
// Neither the loads nor the products alone: without loads 8192^3 took 507 us, without
// products 564 (64 KB a step for 1024 clocks of products); what is missing to the library,
// which reads the same operands, is their overlap.  The tile of 256 columns spills 60 bytes
// a thread (96 registers for 18 warps).  Activations and a second output add their
// epilogue: 98 us with silu and pre-activations for 84, in a graph.  Rows that are no
// multiple of 4 are stored one element a lane: 4096 x 32003 x 2048 486 us, 32000 298.
// 8 tokens on 65536 x 2048: HBM, 45 us = 0.88 of a copy.  33 on 2887 x 2880 8.4 us: latency
// of the launch, one round of steps and the join.  fp32 rows: 4096 x 2048 x 2048 87 us for an
// fp32 result (54 for its three products of parts at the measured rate, the split before
// them 16), 62 for a 16-bit one (two products, 36).
#include <cuda.h>
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "dense.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

using namespace gemm;

// Tile rows of a CTA, k of a step.  (A step's barriers, copies and commit cost the
// issuing threads about 500 clocks: with 64 of k, whose products take 512, 8192^3 took
// 638 us.)
constexpr int kBM = 128, kBK = 128;
constexpr int kChunk32 = 4, kChunk16 = 16;  // steps between drains
constexpr int kWTma = 0, kWMma = 1, kWEpi = 2;
constexpr int kMaxSplits = 8;
constexpr int kChunkMn = kBK * 128;   // bytes of a step's rows of 64 m (n)

// Tiles of 128 x BN to a CTA, or (PAIR) of 256 x BN to the two CTAs of a cluster: each
// has half of A's rows, half of B's and half of the result's, and the leader (rank 0)
// issues the products of both.
template <int BN, bool PAIR>
struct Cfg {
    static constexpr int TM = PAIR ? 2 * kBM : kBM, BR = PAIR ? BN / 2 : BN;  // tile rows; rows of B to a CTA
    static constexpr int EPI = BN >= 128 ? 16 : 8, THREADS = (2 + EPI) * 32;  // epilogue warps
    static constexpr int NC = BN * 4 / EPI, GROUP = NC < 16 ? NC : 16;        // columns of a thread, staged at a time
    static constexpr int A_BYTES = kBM * kBK * 2, B_BYTES = BR * kBK * 2, SLOT = A_BYTES + B_BYTES;
    static constexpr int STAGES = BR == 128 ? 3 : BR == 64 ? 4 : 5;
    static constexpr int STAGING = STAGES * SLOT;      // the epilogue's: GROUP x 32 sums a warp
    static constexpr int BAR_OFF = STAGING + EPI * GROUP * 128;
    static constexpr int MISC_OFF = BAR_OFF + (2 * STAGES + 4) * 8;
    static constexpr int SMEM = MISC_OFF + 16 + 1024;  // (the first 1024: alignment)
    static constexpr int COLS = 2 * BN;                // TMEM: two accumulators
    static_assert(BN * kBM * 4 <= STAGING, "a split tile's sums");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *tm, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst),
        "l"((uint64_t)tm), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Descriptor of a 128-byte swizzled operand.  k contiguous: 8-row groups 1024 bytes
// apart.  m (n) contiguous: chunks of 64 of it `chunk` bytes apart, groups of 8 k 1024.
__device__ __forceinline__ uint64_t descriptor(uint32_t addr, bool mn, uint32_t chunk) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(mn ? chunk >> 4 : 1) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// The same into this CTA of a pair, its bytes counted by a barrier of either CTA.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *tm, int x, int y, int z,
                                                 uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"((uint64_t)tm), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// A shared address of this CTA as that of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t mapped(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrival of a warp, by its lane 0, at a barrier of the cluster.  (Without a release to the
// cluster, which would wait for the last tile's stores; what it orders, reads of TMEM, is
// done.)
__device__ __forceinline__ void arrive_cluster_warp(uint32_t bar, int lane) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.eq.s32 p, %1, 0;\n"
        "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n}" ::"r"(bar),
        "r"(lane)
        : "memory");
}

// One MMA by the converged warp's elected lane.
template <bool PAIR>
__device__ __forceinline__ void mma_warp(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if (PAIR)
        asm volatile(
            "{\n.reg .pred p, e;\nsetp.ne.b32 p, %4, 0;\nelect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p, e;\nsetp.ne.b32 p, %4, 0;\nelect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}
// Arrival at a barrier (of both CTAs of a pair) when the lane's products are done.
template <bool PAIR>
__device__ __forceinline__ void commit_warp(uint32_t bar, int ctas) {
    if (PAIR)
        asm volatile(
            "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}" ::
                "r"(bar),
            "h"((unsigned short)ctas)
            : "memory");
    else
        mma_commit_warp(bar);
}

// A finished sum of lower parts' products.  Not finite, it goes: an infinity times a lower
// part that is zero or of the other sign is not what the formula has; the first parts'
// product holds that infinity, or NaN, times a number of the value's own sign.
__device__ __forceinline__ float lower_sum(float v) { return isfinite(v) ? v : 0.0f; }

struct Tile {
    const DenseProduct *p;
    int m0, n0, kb, first, last;  // kb: steps of one pair of parts; [first, last): this CTA's
    int low, chunk, share;        // low: steps of all pairs but the last, the largest products
    // the step after the last one that is added up in TMEM from step i on
    __device__ __forceinline__ int chunk_end(int i) const {
        return i < low ? min(min(last, low), i + kChunk16) : min(last, i + chunk);
    }
};

// The j-th tile of worker w (a cluster), or false.  Workers take the first product's
// tiles in turn, then the second's (shorter ones) in turn too, but each as many as
// the plan has it: those with fewer of the first take more.  Neighbouring workers are
// at neighbouring tiles; in a product, bands of 8 tiles of m run through all n, so that
// the CTAs at work share rows of both operands in L2.
template <int BN, bool PAIR>
__device__ __forceinline__ bool tile_of(const DenseGemm &g, int worker, int workers, int j, int split, Tile &r) {
    const int one = g.p[0].m_tiles * g.p[0].n_tiles, n0 = one * g.p[0].shares;
    int t = j * workers + worker, of = g.splits;
    r.p = &g.p[0];
    r.share = 0;
    if (t < n0) {
        if (g.p[0].shares > 1) {
            r.share = split = t / one;
            of = g.p[0].shares;
            t -= split * one;
        }
    } else {
        if (g.n_products == 1) return false;
        const int more = n0 % workers, group = worker < more ? 0 : 1, mine = n0 / workers + (group == 0 ? 1 : 0);
        const int k = j - mine, both = min(g.second[0], g.second[1]);
        if (k >= g.second[group]) return false;
        const int members = group == 0 ? more : workers - more, i = group == 0 ? worker : worker - more;
        t = k < both ? k * workers + worker : both * workers + (k - both) * members + i;
        r.p = &g.p[1];
        if (t >= r.p->m_tiles * r.p->n_tiles) return false;
    }
    constexpr int BAND = 8;
    const int band = t / (BAND * r.p->n_tiles), first = band * BAND, size = min(BAND, r.p->m_tiles - first);
    t -= band * BAND * r.p->n_tiles;
    r.m0 = (first + t % size) * Cfg<BN, PAIR>::TM;
    r.n0 = t / size * BN;
    r.kb = (r.p->K + kBK - 1) / kBK;
    const long long steps = (long long)r.kb * r.p->n_pairs;
    r.first = (int)(steps * split / of);
    r.last = (int)(steps * (split + 1) / of);
    r.chunk = r.p->o.dtype == 0 ? kChunk32 : kChunk16;
    r.low = r.kb * (r.p->n_pairs - 1);
    return true;
}

template <int BN, bool PAIR>
__global__ void __launch_bounds__((Cfg<BN, PAIR>::THREADS), 1) dense_gemm_kernel(const __grid_constant__ DenseGemm g) {
    using C = Cfg<BN, PAIR>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    // CTAs of a tile: S (pairs) share out its steps, the two of a pair its rows
    const int S = g.splits, CTAS = PAIR ? 2 * S : S, rank = CTAS > 1 ? (int)cluster.block_rank() : 0;
    const int split = PAIR ? rank >> 1 : rank, side = PAIR ? rank & 1 : 0, leader = rank - side;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t slots = smem_u32(smem), bars = smem_u32(smem + C::BAR_OFF);
    const auto full = [&](int s) { return bars + 8 * s; };
    const auto empty = [&](int s) { return bars + 8 * (C::STAGES + s); };
    const auto acc_full = [&](int b) { return bars + 8 * (2 * C::STAGES + b); };
    const auto acc_empty = [&](int b) { return bars + 8 * (2 * C::STAGES + 2 + b); };
    volatile int *abort_flag = (volatile int *)(smem + C::MISC_OFF);
    uint32_t *tmem_slot = (uint32_t *)(smem + C::MISC_OFF + 4);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), PAIR ? 2 * C::EPI : C::EPI);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (warp == kWMma) {
        if (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(tmem_slot)),
                         "n"(C::COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(tmem_slot)),
                         "n"(C::COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    if (PAIR)
        cluster.sync();  // (both CTAs' barriers are ready before either is signalled)
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // (worked out anew each time: the epilogue has no registers to keep it in)
    const auto tile = [&](int j, Tile &w) {
        return tile_of<BN, PAIR>(g, (int)blockIdx.x / CTAS, (int)gridDim.x / CTAS, j, split, w);
    };

    if (warp == kWTma) {
        if (lane == 0) {
            // (parts that the kernel before wrote are read by the copies' proxy)
            asm volatile("fence.proxy.async;" ::: "memory");
            // the leader's barriers count both CTAs' bytes
            const uint32_t full_at = PAIR ? mapped(full(0), leader) : full(0);
            uint32_t it = 0, slot = 0, phase = 0;
            Tile w;
            for (int j = 0; tile(j, w); ++j) {
                // (what a step needs in registers: a load of the parameters costs each step more
                // than its copies' issue)
                const bool a_mn = w.p->a_mn, b_mn = w.p->b_mn, fold = w.p->fold;
                const CUtensorMap *tm_a = &w.p->tm_a, *tm_b = &w.p->tm_b;
                const int m0 = w.m0 + side * kBM, n0 = w.n0 + side * C::BR, k_end = w.kb * kBK;
                int k = w.first % w.kb * kBK;
                unsigned pairs = w.p->pairs >> (4 * (w.first / w.kb));
                for (int i = w.first; i < w.last; ++i, ++it) {
                    if (!mbar_wait(empty(slot), phase ^ 1, abort_flag, g.error, kErrorDense)) goto loaded;
                    const uint32_t a = slots + slot * C::SLOT, b = a + C::A_BYTES, bar = full_at + 8 * slot;
                    const int part_a = pairs & 3, part_b = pairs >> 2 & 3;
                    if (side == 0) mbar_arrive_tx(full(slot), PAIR ? 2 * C::SLOT : C::SLOT);
                    const auto load = [&](uint32_t dst, const CUtensorMap *tm, int x, int y, int z) {
                        if (PAIR)
                            tma_load_3d_pair(dst, tm, x, y, z, bar);
                        else
                            tma_load_3d(dst, tm, x, y, z, bar);
                    };
                    if (a_mn) {
                        load(a, tm_a, m0, k, part_a);
                        load(a + C::A_BYTES / 2, tm_a, m0 + 64, k, part_a);
                    } else {
                        load(a, tm_a, k, m0, part_a);
                        load(a + C::A_BYTES / 2, tm_a, k + 64, m0, part_a);
                    }
                    if (fold) {
                        load(b, tm_b, k, 0, n0 / 4);
                        load(b + C::B_BYTES / 2, tm_b, k + 64, 0, n0 / 4);
                    } else if (C::BR >= 64 && b_mn) {
#pragma unroll
                        for (int c = 0; c < C::BR / 64; ++c) load(b + c * kChunkMn, tm_b, n0 + 64 * c, k, part_b);
                    } else {
                        load(b, tm_b, k, n0, part_b);
                        load(b + C::B_BYTES / 2, tm_b, k + 64, n0, part_b);
                    }
                    k += kBK;
                    if (k == k_end) {
                        k = 0;
                        pairs >>= 4;
                    }
                    if (++slot == C::STAGES) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
            // no CTA ends before the arrivals at its last stages have come
            for (uint32_t i = it > C::STAGES ? it - C::STAGES : 0; i < it; ++i)
                if (!mbar_wait(empty(i % C::STAGES), i / C::STAGES & 1, abort_flag, g.error, kErrorDense)) break;
        loaded:;
        }
        __syncwarp();
    } else if (warp == kWMma) {
        uint32_t slot = 0, phase = 0, chunk = 0;
        Tile w;
        for (int j = 0; side == 0 && tile(j, w); ++j) {
            const bool a_mn = w.p->a_mn, b_mn = w.p->b_mn;
            // fp32 sums, both operands binary16 (0) or bfloat16 (1), their directions, N, M
            const uint32_t type = w.p->bf16 ? 1u : 0u;
            const uint32_t idesc = (1u << 4) | type << 7 | type << 10 | (a_mn ? 1u << 15 : 0) | (b_mn ? 1u << 16 : 0) |
                                   (uint32_t)(BN >> 3) << 17 | (uint32_t)(C::TM >> 4) << 24;
            const uint64_t a0 = descriptor(slots, a_mn, kChunkMn), b0 = descriptor(slots + C::A_BYTES, b_mn, kChunkMn);
            // 16 of k: 32 bytes in a row of 64 k (and the second block), 16 rows of 128 bytes
            // in the other kind
            const uint32_t a_step = (a_mn ? 2048 : 32) >> 4, a_half = (a_mn ? 8192 : C::A_BYTES / 2) >> 4;
            const uint32_t b_step = (b_mn ? 2048 : 32) >> 4, b_half = (b_mn ? 8192 : C::B_BYTES / 2) >> 4;
            for (int i = w.first; i < w.last; ++chunk) {
                const int buf = chunk & 1, end = w.chunk_end(i);
                if (!mbar_wait_warp(acc_empty(buf), (chunk >> 1 & 1) ^ 1, abort_flag, g.error, kErrorDense)) goto multiplied;
                tc_fence_after();
                const uint32_t d = tmem + buf * BN;
                uint32_t more = 0;
                for (; i < end; ++i) {
                    if (!mbar_wait_warp(full(slot), phase, abort_flag, g.error, kErrorDense)) goto multiplied;
                    tc_fence_after();
                    const uint32_t at = slot * (C::SLOT >> 4);
#pragma unroll
                    for (int q = 0; q < kBK / 16; ++q) {
                        mma_warp<PAIR>(d, a0 + at + q % 4 * a_step + q / 4 * a_half,
                                       b0 + at + q % 4 * b_step + q / 4 * b_half, idesc, more);
                        more = 1;
                    }
                    commit_warp<PAIR>(empty(slot), 3 << leader);
                    if (++slot == C::STAGES) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                commit_warp<PAIR>(acc_full(buf), 3 << leader);
            }
        }
    multiplied:;
        __syncwarp();
    } else {
        // lanes of TMEM: a warp reaches the quarter of its number
        const int quarter = warp & 3, share = (warp - kWEpi) >> 2;
        constexpr int NC = C::NC, GROUP = C::GROUP;
        // (the first products are some time off)
        if (g.sums)
            dense::finish_sums(g.sum_parts, g.sums, g.sum_blocks, g.sum_cols,
                               (int)blockIdx.x + (int)gridDim.x * (warp - kWEpi), (int)gridDim.x * C::EPI, lane);
        uint32_t chunk = 0;
        Tile w;
        for (int j = 0; tile(j, w); ++j) {
            float acc[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[c] = 0.0f;
            for (int i = w.first, end; i < w.last; i = end, ++chunk) {
                const int buf = chunk & 1;
                end = w.chunk_end(i);
                if (!mbar_wait_warp(acc_full(buf), chunk >> 1 & 1, abort_flag, g.error, kErrorDense)) goto finished;
                tc_fence_after();
                const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + buf * BN + share * NC;
#pragma unroll
                for (int c = 0; c < NC; c += 16) {
                    uint32_t v[16];
                    tmem_ld16u(at + c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[c + j] += __uint_as_float(v[j]);
                }
                // (the lower parts' products come first)
                if (i < w.low && end == min(w.last, w.low))
#pragma unroll
                    for (int c = 0; c < NC; ++c) acc[c] = lower_sum(acc[c]) * w.p->low_scale;
                tc_fence_before();
                if (PAIR)
                    arrive_cluster_warp(mapped(acc_empty(buf), leader), lane);
                else
                    mbar_arrive_warp(acc_empty(buf), lane);
            }
            const int ml = quarter * 32 + lane, n0 = w.n0 + share * NC, m = w.m0 + side * kBM + ml;
            const float bias = S == 1 && w.p->o.bias && m < w.p->M ? w.p->o.bias[m] : 0.0f, scale = w.p->scale;
            if (S > 1) {
                // (all products of the CTA are done: its stages are free)
                float *red = (float *)smem;
#pragma unroll
                for (int c = 0; c < NC; ++c) red[(share * NC + c) * kBM + ml] = acc[c] * scale;
            } else if (w.p->fold) {
                const dense::Epilogue e(w.p->o, w.p->M, w.m0 + side * kBM + quarter * 32 + (lane & 7) * 4, 0);
                float *mine = (float *)(smem + C::STAGING) + (warp - kWEpi) * GROUP * 32;
                // (the lowest parts first)
#pragma unroll
                for (int c = 0; c < NC; c += 4 * GROUP) {
                    constexpr int TOKENS = NC / 4 < GROUP ? NC / 4 : GROUP;
#pragma unroll
                    for (int j = 0; j < TOKENS; ++j)
                        mine[j * 32 + lane] = lower_sum(acc[c + 4 * j + 2] + acc[c + 4 * j + 1]) + acc[c + 4 * j] + bias;
                    __syncwarp();
                    e.store(mine, TOKENS, (n0 + c) / 4, w.p->N / 4, lane);
                    __syncwarp();
                }
            } else {
                const dense::Epilogue e(w.p->o, w.p->M, w.m0 + side * kBM + quarter * 32 + (lane & 7) * 4,
                                        (size_t)w.share * w.p->M * w.p->N);
                float *mine = (float *)(smem + C::STAGING) + (warp - kWEpi) * GROUP * 32;
#pragma unroll
                for (int c = 0; c < NC; c += GROUP) {
#pragma unroll
                    for (int j = 0; j < GROUP; ++j) mine[j * 32 + lane] = fmaf(acc[c + j], scale, bias);
                    __syncwarp();
                    e.store(mine, GROUP, n0 + c, w.p->N, lane);
                    __syncwarp();
                }
            }
        }
    finished:;
        __syncwarp();
    }
    __syncthreads();
    if (S > 1) {
        cluster.sync();
        if (!*abort_flag) {
            // a lane: four rows; a warp: a column; the CTAs of the same rows: every S-th warp
            Tile w;
            tile(0, w);
            const dense::Epilogue e(w.p->o, w.p->M, w.m0 + side * kBM + lane * 4, 0);
            const float4 *red = (const float4 *)smem + lane;
            float bias[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) bias[j] = e.o.bias && j < e.left ? e.o.bias[e.m + j] : 0.0f;
            const int fold = w.p->fold ? 4 : 1, cols = min(BN, w.p->N - w.n0) / fold;
            for (int c = split * (C::THREADS / 32) + warp; c < cols; c += S * (C::THREADS / 32)) {
                float sum[4] = {};
                for (int f = fold > 1 ? 2 : 0; f >= 0; --f) {  // (the lowest parts first, the fourth is zero)
                    if (f == 0)
#pragma unroll
                        for (int j = 0; j < 4; ++j) sum[j] = lower_sum(sum[j]);
                    float4 v[kMaxSplits];
#pragma unroll
                    for (int s = 0; s < kMaxSplits; ++s)
                        if (s < S)
                            v[s] = *cluster.map_shared_rank(red + (c * fold + f) * (kBM / 4), PAIR ? 2 * s + side : s);
#pragma unroll
                    for (int s = 0; s < kMaxSplits; ++s)
                        if (s < S) sum[0] += v[s].x, sum[1] += v[s].y, sum[2] += v[s].z, sum[3] += v[s].w;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] += bias[j];
                if (e.left > 0) e.column(sum, w.n0 / fold + c);
            }
        }
        __syncwarp();
        cluster.sync();  // no CTA leaves while its sums are read
    }
    // after an abort, give the copies and MMAs of this CTA a bounded time (about 10 ms)
    // to land, then free TMEM
    if (*abort_flag) {
        const long long t0 = clock64();
        while (clock64() - t0 < 20000000ll) {
        }
    }
    tc_fence_before();
    if (PAIR)
        cluster.sync();  // no CTA leaves while the other's products read it or its arrivals come
    else
        __syncthreads();
    tc_fence_after();
    if (warp == kWMma) {
        if (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::COLS) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::COLS) : "memory");
    }
}

long long steps_of(const DenseProduct &p) { return (long long)((p.K + kBK - 1) / kBK) * p.n_pairs; }

// Tiles of a second product (n1 of s1 steps) for the workers that have one tile more of
// the first (n0 of s0) and for the others, so that the longest is as short as it can be:
// its steps.
long long share_out(long long n0, long long s0, long long n1, long long s1, long long workers, int *second) {
    const long long more = n0 % workers, low = n0 / workers * s0, high = low + s0;
    const auto fits = [&](long long level, long long load) { return level > load ? (level - load) / s1 : 0; };
    const auto room = [&](long long level) { return more * fits(level, high) + (workers - more) * fits(level, low); };
    // between an even share of all and what the last tiles may add to it
    long long from = (n0 * s0 + n1 * s1) / workers, to = std::max(from, high) + s0 + s1;
    while (from < to) {
        const long long level = (from + to) / 2;
        if (room(level) >= n1)
            to = level;
        else
            from = level + 1;
    }
    if (second) {
        second[0] = (int)fits(to, high);
        second[1] = (int)fits(to, low);
    }
    return std::max(to, more > 0 ? high : low);
}


// The tiles that are compiled, and what one costs.  Clocks of a step: measured, but
// for the pairs' near what 128 bytes a clock of shared memory allow (a step's operands
// are written there once and read once; a pair's B is read by halves).
struct Shape {
    int bn;
    bool pair;
    double clocks;
};
constexpr Shape kShapes[] = {
    {256, true, 1120}, {128, true, 840}, {128, false, 1280}, {64, false, 960}, {32, false, 840}};

template <int BN, bool PAIR>
int launch_tile(DenseGemm &g, int device, int n_sm, cudaStream_t st) {
    using C = Cfg<BN, PAIR>;
    auto kernel = dense_gemm_kernel<BN, PAIR>;
    static std::atomic<unsigned long long> configured{0};  // a bit a device
    if (!(configured.load() >> (device & 63) & 1)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return (int)e;
        configured.fetch_or(1ull << (device & 63));
    }
    for (int i = 0; i < g.n_products; ++i) {
        DenseProduct &p = g.p[i];
        p.m_tiles = (p.M + C::TM - 1) / C::TM;
        p.n_tiles = (p.N + BN - 1) / BN;
    }
    const int ctas = PAIR ? 2 * g.splits : g.splits, n0 = g.p[0].m_tiles * g.p[0].n_tiles * g.p[0].shares;
    const int n1 = g.n_products > 1 ? g.p[1].m_tiles * g.p[1].n_tiles : 0;
    const int workers = g.splits > 1 ? n0 : std::min(n0 + n1, n_sm / ctas);
    if (n1 > 0) share_out(n0, (steps_of(g.p[0]) + g.p[0].shares - 1) / g.p[0].shares, n1, steps_of(g.p[1]), workers, g.second);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)workers * ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)ctas, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return (int)cudaLaunchKernelEx(&cfg, kernel, g);
}

// Clusters of `ctas` CTAs that run at a time (a GPC's SMs that make up no whole cluster
// stay idle: 76 of 2, 46 of 3, 36 of 4, 23 of 6 and 15 of 8 on 152 SMs).
int clusters_at_once(int ctas, int device, int n_sm) {
    if (ctas == 1) return n_sm;
    static std::atomic<int> known[64][kMaxSplits + 1];  // 0: not asked yet
    std::atomic<int> &n = known[device & 63][ctas];
    if (n.load() == 0) {
        using C = Cfg<256, true>;  // (one CTA of any tile fills an SM)
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)ctas);
        cfg.blockDim = dim3(C::THREADS);
        cfg.dynamicSmemBytes = C::SMEM;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {(unsigned)ctas, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int most = 0;
        if (cudaFuncSetAttribute(dense_gemm_kernel<256, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
                cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&most, dense_gemm_kernel<256, true>, &cfg) != cudaSuccess || most < 1) {
            cudaGetLastError();
            most = std::max(1, n_sm / ctas / 2);
        }
        n.store(most);
    }
    return n.load();
}

}  // namespace

// The cheapest of the tiles and K splits, by the clocks of the longest CTA.  (A model, right
// where tiles fill the SMs and to 7% for few tokens; for split pairs it counts the join too
// low: 512 tokens on 4096 x 4096 22.4 us with the 256p/2 it takes, 19.2 with 128p/1; 2048 on
// 512 x 2048 12.5 with 128p/2, 10.3 with 64/1.)
DensePlan dense_plan(const DenseProduct *p, int n_products, int device, int n_sm) {
    DensePlan best{};
    for (const Shape &f : kShapes) {
        const int tm = f.pair ? 2 * kBM : kBM;
        bool fits = true;
        long long tiles[2] = {}, steps[2] = {};  // (of a tile)
        for (int i = 0; i < n_products; ++i) {
            if (p[i].b_mn && (f.pair ? f.bn / 2 : f.bn) < 64) fits = false;  // (columns of B come 64 at a time)
            tiles[i] = (long long)((p[i].M + tm - 1) / tm) * ((p[i].N + f.bn - 1) / f.bn);
            steps[i] = steps_of(p[i]);
        }
        if (!fits) continue;
        const auto consider = [&](int splits, int shares) {
            const int workers = clusters_at_once(f.pair ? 2 * splits : splits, device, n_sm);
            const long long n0 = tiles[0] * shares, s0 = (steps[0] + splits * shares - 1) / (splits * shares);
            const long long rounds = (n0 + workers - 1) / workers;
            if (splits > 1 && rounds > 1) return;
            const long long longest =
                n_products == 1 ? rounds * s0
                                : share_out(n0, s0, tiles[1], steps[1], std::min<long long>(n0 + tiles[1], workers), nullptr);
            // joins: through shared memory, or through HBM at its rate
            const double c = (double)longest * f.clocks + (splits > 1 ? 2500 + 20 * f.bn : 12 * f.bn) +
                             (shares > 1 ? 6000 + 1.5e-3 * p[0].M * p[0].N * shares : 0);
            if (best.splits == 0 || c < best.clocks) best = {f.bn, f.pair ? f.bn / 2 : f.bn, f.pair, splits, shares, c};
        };
        if (n_products == 1)
            for (int s = 1; s <= std::min<long long>(f.pair ? kMaxSplits / 2 : kMaxSplits, steps[0]); ++s) consider(s, 1);
        for (int s = n_products == 1 ? 2 : 1; s <= std::min<long long>(std::max(1, p[0].most_shares), steps[0]); ++s)
            consider(1, s);
    }
    return best;
}

int dense_steps(const DenseProduct &p) { return (int)std::min(steps_of(p), 1ll << 30); }

int launch_dense_gemm(DenseGemm &g, const DensePlan &plan, int device, int n_sm, cudaStream_t st) {
    if (plan.pair)
        return plan.bn == 256 ? launch_tile<256, true>(g, device, n_sm, st) : launch_tile<128, true>(g, device, n_sm, st);
    switch (plan.bn) {
        case 32: return launch_tile<32, false>(g, device, n_sm, st);
        case 64: return launch_tile<64, false>(g, device, n_sm, st);
        default: return launch_tile<128, false>(g, device, n_sm, st);
    }
}

}  // namespace moe
