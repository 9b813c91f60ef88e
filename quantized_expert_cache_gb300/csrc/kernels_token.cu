// Log probabilities of given tokens, the entropy and the largest logits of a
// row over the vocabulary, and the gradient of the first two.
//
//   z = scale x,  m = max x,  u_j = scale (x_j - m),  S = sum_j exp(u_j)
//   logp_j = u_j - log S,   H = log S - sum_j exp(u_j) u_j / S
//   dx_j = scale (g [j = target] - p_j (g + g_H (logp_j + H)))
//
// One pass over the row.  A warp keeps one running maximum for its lanes, so
// sums are rescaled only when a tile of its elements passes it, and the sums of
// warps and CTAs are joined at the end.  The elements equal to the maximum are
// counted, not summed: S - 1 keeps its own 24 bits, and log S = log1p(S - 1) and H
// are right to their last digits for a row of one likely token too.  All terms of H
// are positive.
//
// The n largest: the row falls into at most 256 units, whose maxima the pass
// keeps anyway.  The n-th largest of these is a bound below the n-th largest
// element, and units below it hold none of the n; the others, about n of them, are
// read again (from L2) into lists of 32 sorted over a warp's lanes, which are merged
// pairwise.  Keys hold the value over the inverted index, so order and ties (the
// lowest index) are one comparison of whole numbers, whatever the order of work.
//
// A row takes a cluster of 1 to 16 CTAs, joined through distributed shared memory:
// no workspace, any stream, one launch.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kTokenWarps = kThreads / 32;
constexpr int kTokenCluster = 8, kTokenGradPacks = 4;
constexpr int kUnits = 256;   // units of a row at most: one thread each for their order
constexpr int kList = 32;     // entries of a sorted list, one a lane
constexpr float kInf = __builtin_inff();
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
static_assert(kTokenMaxTop <= kList, "a list holds the largest n_top");

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

template <typename T>
struct alignas(16) Pack16 {
    static constexpr int N = 16 / sizeof(T);
    T v[N];
};

// 2^x for x <= 0 by the special-function unit; NaN stays.
__device__ __forceinline__ float exp2_neg(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// The larger, NaN if either is: exponents below -200 (and -infinity) give 2^x = 0
// and 2^x x = 0, a NaN stays one.
__device__ __forceinline__ float bounded(float x) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(-200.0f));
    return r;
}

// Whole numbers that order like the values (+0 and -0 alike), and back.
__device__ __forceinline__ unsigned order_of(float x) {
    const unsigned b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_order(unsigned k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// Sums of a set of elements relative to its largest, m: `s` of 2^u, `n` the count
// of u = 0 left out of it, `t` the sum of 2^u u.
struct Sums {
    float m, s, n, t;
};

// Sums relative to a larger maximum, d = c (m - new) <= 0 in units of log2.
__device__ __forceinline__ void lower(Sums &a, float d) {
    const float f = exp2_neg(bounded(d)), all = a.s + a.n;
    a.t = f * (a.t + bounded(d) * all);
    a.s = f * all;
    a.n = 0.0f;
}
__device__ __forceinline__ Sums joined(Sums a, Sums b, float c) {
    const float m = fmaxf(a.m, b.m);
    // (an empty set's m is -infinity, its sums 0 or NaN; so no d is NaN)
    if (a.m != m) lower(a, a.m == -kInf ? -kInf : c * (a.m - m));
    if (b.m != m) lower(b, b.m == -kInf ? -kInf : c * (b.m - m));
    return Sums{m, a.s + b.s, a.n + b.n, a.t + b.t};
}

// A row as packs of 16 bytes from the boundary at or below its first element:
// element j of pack i is the row's element i N + j - head.
template <typename T>
struct Row {
    const T *x;
    int head, vocab;
    __device__ __forceinline__ Row(const void *logits, size_t row, int vocab_)
        : x((const T *)logits + row * (size_t)vocab_), vocab(vocab_) {
        head = (int)(((uintptr_t)x & 15) / sizeof(T));
    }
    __device__ __forceinline__ Pack16<T> load(int pack) const {
        constexpr int N = Pack16<T>::N;
        const int e = pack * N - head;
        if (e >= 0 && e + N <= vocab) return *(const Pack16<T> *)(x + e);
        Pack16<T> p;
#pragma unroll
        for (int j = 0; j < N; ++j) p.v[j] = e + j >= 0 && e + j < vocab ? x[e + j] : rounded<T>(-kInf);
        return p;
    }
};

// Two sorted lists (largest in lane 0) -> the 32 largest of both, sorted.
__device__ __forceinline__ unsigned long long merge32(unsigned long long a, unsigned long long b, int lane) {
    const unsigned long long r = __shfl_sync(0xffffffffu, b, 31 - lane);
    a = a > r ? a : r;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long q = __shfl_xor_sync(0xffffffffu, a, o);
        a = (lane & o) == 0 ? (a > q ? a : q) : (a < q ? a : q);
    }
    return a;
}

// The sums of lanes 0 to WIDTH - 1 (the others' ignored) in all of these, joined in
// a fixed tree: the same bits whatever the order that warps and CTAs ran in.
template <int WIDTH>
__device__ __forceinline__ Sums joined_lanes(Sums q, float c) {
#pragma unroll
    for (int o = 1; o < WIDTH; o <<= 1)
        q = joined(q,
                   Sums{__shfl_xor_sync(0xffffffffu, q.m, o), __shfl_xor_sync(0xffffffffu, q.s, o),
                        __shfl_xor_sync(0xffffffffu, q.n, o), __shfl_xor_sync(0xffffffffu, q.t, o)},
                   c);
    return q;
}

// The kTokenWarps lists of a CTA's warps (lists[warp], each lane's entry in `list`)
// -> the largest 32 of all in warp 0.
__device__ __forceinline__ unsigned long long merge_warps(unsigned long long (*lists)[kList], unsigned long long list,
                                                          int warp, int lane) {
    lists[warp][lane] = list;
    for (int n = kTokenWarps / 2; n > 0; n >>= 1) {
        __syncthreads();
        if (warp < n) lists[warp][lane] = list = merge32(list, lists[warp + n][lane], lane);
    }
    return list;
}

struct TokenShared {
    Sums part[kTokenWarps];           // of the warps
    Sums cta;
    unsigned unit[kUnits];            // the maxima of this CTA's units
    unsigned all[kUnits];             // of all CTAs'
    unsigned long long list[kTokenWarps][kList], joint[kTokenWarps][kList];
    int flagged[kUnits];
    int n_flagged;
    unsigned bound;  // 0: every unit may hold one
};

// U packs a lane and tile; a unit is 2^shift tiles of a warp.
template <typename T, int U>
__global__ void __launch_bounds__(kThreads, 4) token_logprobs_kernel(TokenParams p, int shift, int units_cta) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int N = Pack16<T>::N, TILE = 32 * U;  // packs of a tile
    __shared__ TokenShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t row = blockIdx.x / C;
    const Row<T> r(p.logits, row, p.vocab);
    const int packs = (r.head + p.vocab + N - 1) / N;
    const int units = (packs + (TILE << shift) - 1) / (TILE << shift);
    const int u0 = min(units, rank * units_cta), u1 = min(units, u0 + units_cta);
    const float c = p.scale * kLog2e;

    // one thread of the row writes its results
    int target = -1;
    float x_target = 0.0f;
    if (rank == 0 && threadIdx.x == 0) {
        target = p.targets ? p.targets[row] : -1;
        if (target >= p.vocab) {
            atomicOr(p.error, kErrorToken);
            target = -1;
        }
        if (target >= 0) x_target = value<T>(r.x[target]);
    }

    // ---- the pass: tiles in turn, the next one's loads in flight
    Sums a{-kInf, 0.0f, 0.0f, 0.0f};
    const int mine = u0 + warp < u1 ? (u1 - u0 - warp + kTokenWarps - 1) / kTokenWarps : 0;
    const int tiles = mine << shift;
    auto tile_pack = [&](int i) {
        const int unit = u0 + warp + (i >> shift) * kTokenWarps;
        return ((unit << shift) + (i & ((1 << shift) - 1))) * TILE + lane;
    };
    Pack16<T> next[U];
    if (tiles > 0)
#pragma unroll
        for (int k = 0; k < U; ++k) next[k] = r.load(tile_pack(0) + 32 * k);
    unsigned top = 0;
    for (int i = 0; i < tiles; ++i) {
        float x[U * N];
        float high = -kInf;
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                x[k * N + j] = value<T>(next[k].v[j]);
                high = fmaxf(high, x[k * N + j]);
            }
        if (i + 1 < tiles) {
            const int at = tile_pack(i + 1);
#pragma unroll
            for (int k = 0; k < U; ++k) next[k] = r.load(at + 32 * k);
        }
        const unsigned key = __reduce_max_sync(0xffffffffu, order_of(high));
        const float tm = of_order(key);
        top = max(top, key);
        if ((i & ((1 << shift) - 1)) == (1 << shift) - 1) {
            if (lane == 0) sh.unit[warp + (i >> shift) * kTokenWarps] = top;
            top = 0;
        }
        if (tm > a.m) {
            if (a.m != -kInf) lower(a, c * (a.m - tm));
            a.m = tm;
        }
        // (all -infinity so far: relative to 0 they stay it)
        const float m = a.m == -kInf ? 0.0f : a.m;
        if (tm < a.m) {
#pragma unroll
            for (int e = 0; e < U * N; ++e) {
                const float u = bounded((x[e] - m) * c), f = exp2_neg(u);
                a.s += f;
                a.t = fmaf(f, u, a.t);
            }
        } else {
#pragma unroll
            for (int e = 0; e < U * N; ++e) {
                const float u = bounded((x[e] - m) * c), f = exp2_neg(u);
                const bool is_max = u == 0.0f;
                a.n += is_max ? 1.0f : 0.0f;
                a.s += is_max ? 0.0f : f;
                a.t = fmaf(f, u, a.t);
            }
        }
    }
    a.s = warp_sum_f(a.s);
    a.n = warp_sum_f(a.n);
    a.t = warp_sum_f(a.t);
    if (lane == 0) sh.part[warp] = a;
    if (threadIdx.x == 0) sh.n_flagged = 0, sh.bound = 0;
    __syncthreads();
    if (warp == 0) {
        a = joined_lanes<kTokenWarps>(sh.part[lane % kTokenWarps], c);
        if (lane == 0) sh.cta = a;
    }
    if (C > 1)
        cluster.sync();
    else
        __syncthreads();

    // ---- the units that may hold one of the n largest
    unsigned long long best = 0;  // rank 0, warp 0: lane i's is the i-th largest
    if (p.n_top > 0) {
        unsigned mine_key = 0;
        const int t = threadIdx.x;
        if (t < units)
            mine_key = C > 1 ? cluster.map_shared_rank(sh.unit, t / units_cta)[t % units_cta] : sh.unit[t];
        sh.all[t] = mine_key;
        __syncthreads();
        if (units > p.n_top) {
            // the maximum with n_top - 1 before it bounds the n largest from below
            int before = 0;
            for (int j = 0; j < units; ++j) {
                const unsigned k = sh.all[j];
                before += k > mine_key || (k == mine_key && j < t) ? 1 : 0;
            }
            if (t < units && before == p.n_top - 1) sh.bound = mine_key;
            __syncthreads();
        }
        const unsigned bound = sh.bound;
        if (t >= u0 && t < u1 && mine_key >= bound) sh.flagged[atomicAdd(&sh.n_flagged, 1)] = t;
        __syncthreads();
        unsigned long long list = 0, last = 0;  // last: the n_top-th entry
        const int n_flagged = sh.n_flagged;
        for (int f = warp; f < n_flagged; f += kTokenWarps) {
            const int first = (sh.flagged[f] << shift) * TILE;
            for (int i = first; i < first + (TILE << shift); i += TILE) {
                Pack16<T> v[U];
#pragma unroll
                for (int k = 0; k < U; ++k) v[k] = r.load(i + 32 * k + lane);
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int e0 = (i + 32 * k + lane) * N - r.head;
                    float high = value<T>(v[k].v[0]);
                    bool nan = high != high;
#pragma unroll
                    for (int j = 1; j < N; ++j) {
                        const float y = value<T>(v[k].v[j]);
                        high = fmaxf(high, y);
                        nan |= y != y;
                    }
                    if (!__any_sync(0xffffffffu, nan || order_of(high) >= bound)) continue;
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const int e = e0 + j;
                        const unsigned key = order_of(value<T>(v[k].v[j]));
                        unsigned long long cand = 0;
                        if (e >= 0 && e < p.vocab && key >= bound)
                            cand = (unsigned long long)key << 32 | (0xffffffffu - (unsigned)e);
                        unsigned who = __ballot_sync(0xffffffffu, cand > last);
                        while (who) {
                            const unsigned long long one = __shfl_sync(0xffffffffu, cand, __ffs(who) - 1);
                            who &= who - 1;
                            if (one > last) {
                                const int at = __popc(__ballot_sync(0xffffffffu, list > one));
                                const unsigned long long up = __shfl_up_sync(0xffffffffu, list, 1);
                                list = lane < at ? list : lane == at ? one : up;
                                last = __shfl_sync(0xffffffffu, list, p.n_top - 1);
                            }
                        }
                    }
                }
            }
        }
        list = merge_warps(sh.list, list, warp, lane);
        if (C > 1) {
            cluster.sync();
            if (rank == 0)  // (C <= kTokenWarps: a warp takes a CTA's list)
                list = merge_warps(sh.joint, warp < C ? cluster.map_shared_rank(sh.list[0], warp)[lane] : 0, warp,
                                   lane);
        }
        best = list;
    }
    // ---- results
    if (rank == 0 && warp == 0) {
        static_assert(kTokenCluster <= kTokenWarps, "one lane and one warp to a CTA");
        Sums q = sh.cta;
        if (C > 1) {
            q = lane % kTokenWarps < C ? *cluster.map_shared_rank(&sh.cta, lane % kTokenWarps)
                                       : Sums{-kInf, 0.0f, 0.0f, 0.0f};
            q = joined_lanes<kTokenWarps>(q, c);
        }
        // nothing but -infinity: no distribution
        const bool none = q.m == -kInf && q.s == 0.0f;
        const float rest = q.s + (q.n - 1.0f);
        const float log_sum = none ? 0.0f : log1pf(rest);
        if (lane == 0) {
            if (p.logp)
                p.logp[row] = target < 0 ? 0.0f : none ? -kInf : (x_target - q.m) * p.scale - log_sum;
            if (p.entropy) p.entropy[row] = none ? 0.0f : log_sum - kLn2 * q.t / (1.0f + rest);
            if (p.stats) {
                p.stats[2 * row] = q.m;
                p.stats[2 * row + 1] = log_sum;
            }
        }
        if (lane < p.n_top) {
            p.top_idx[row * p.n_top + lane] = (int32_t)(0xffffffffu - (unsigned)best);
            const float x = of_order((unsigned)(best >> 32));
            p.top_logp[row * p.n_top + lane] = none ? -kInf : (x - q.m) * p.scale - log_sum;
        }
    }
    if (C > 1) cluster.sync();  // no CTA leaves while its shared memory is read
}

// ---- gradient: one read, one write, a row's scalars in every thread --------------
// CTAs take `step` packs of a row each.  Results go where the logits were, to the
// same thread, when the two buffers are one.
template <typename T>
__global__ void __launch_bounds__(kThreads) token_grad_kernel(TokenGradParams p, int chunks, bool same_align) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int N = Pack16<T>::N;
    const size_t row = blockIdx.x / chunks;
    const Row<T> r(p.logits, row, p.vocab);
    T *dx = (T *)p.dlogits + row * (size_t)p.vocab;
    const int first = (int)(blockIdx.x % chunks) * (kThreads * kTokenGradPacks) + threadIdx.x;
    Pack16<T> v[kTokenGradPacks];
#pragma unroll
    for (int k = 0; k < kTokenGradPacks; ++k) v[k] = r.load(first + kThreads * k);
    int target = p.targets ? p.targets[row] : -1;
    if (target >= p.vocab) {
        if (threadIdx.x == 0) atomicOr(p.error, kErrorToken);
        target = -1;
    }
    const float top = p.stats[2 * row], log_sum = p.stats[2 * row + 1];
    const float g = p.g_logp && target >= 0 ? p.g_logp[row] : 0.0f;
    const float gh = p.g_entropy ? p.g_entropy[row] : 0.0f, h = p.g_entropy ? p.entropy[row] : 0.0f;
    const bool none = top == -kInf && log_sum == 0.0f;
#pragma unroll
    for (int k = 0; k < kTokenGradPacks; ++k) {
        const int e = (first + kThreads * k) * N - r.head;
        if (e + N <= 0 || e >= p.vocab) continue;
        Pack16<T> o;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float lp = (value<T>(v[k].v[j]) - top) * p.scale - log_sum;
            const float q = exp2_neg(bounded(lp * kLog2e));
            // (where q is 0 the clamped factor stays finite)
            float d = -q * gh * (fmaxf(lp, -150.0f) + h);
            // g (1 - p): a likely target's keeps its digits
            d += e + j == target ? -g * expm1f(lp) : -q * g;
            o.v[j] = rounded<T>(none ? 0.0f : d * p.scale);
        }
        if (same_align && e >= 0 && e + N <= p.vocab) {
            *(Pack16<T> *)(dx + e) = o;
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (e + j >= 0 && e + j < p.vocab) dx[e + j] = o.v[j];
        }
    }
}

template <typename K, typename... A>
int launch(K kernel, size_t grid, int cluster, cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return (int)cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int U>
int launch_logprobs(const TokenParams &p, int n_sm, cudaStream_t st) {
    constexpr int N = 16 / (int)sizeof(T), TILE = 32 * U;
    const int packs = (p.vocab + N - 1) / N + 1;  // with any head
    int shift = 0;
    while ((packs + (TILE << shift) - 1) / (TILE << shift) > kUnits) ++shift;
    const int units = (packs + (TILE << shift) - 1) / (TILE << shift);
    // CTAs of a row: as many as keep every warp at a unit, up to four CTAs a SM
    int C = 1;
    while (C < kTokenCluster && (long long)p.n_tokens * C * 2 <= 4ll * n_sm && units >= 2 * C * kTokenWarps) C *= 2;
    auto kernel = token_logprobs_kernel<T, U>;
    return launch(kernel, (size_t)p.n_tokens * C, C, st, p, shift, (units + C - 1) / C);
}

template <typename T>
int launch_rows(const TokenParams &p, int n_sm, cudaStream_t st) {
    // tiles of one pack a lane where that makes no more than kUnits units, else of 16
    // elements a lane
    constexpr int N = 16 / (int)sizeof(T);
    return p.vocab + 16 <= 32 * kUnits * N ? launch_logprobs<T, 1>(p, n_sm, st)
                                           : launch_logprobs<T, 16 / N>(p, n_sm, st);
}

template <typename T>
int launch_grad(const TokenGradParams &p, cudaStream_t st) {
    constexpr int N = 16 / (int)sizeof(T);
    const int packs = (p.vocab + N - 1) / N + 1, chunks = (packs + kThreads * kTokenGradPacks - 1) / (kThreads * kTokenGradPacks);
    return launch(token_grad_kernel<T>, (size_t)p.n_tokens * chunks, 1, st, p, chunks,
                  (((uintptr_t)p.logits ^ (uintptr_t)p.dlogits) & 15) == 0);
}

}  // namespace

int launch_token_logprobs(const TokenParams &p, int n_sm, cudaStream_t st) {
    switch (p.dtype) {
        case 1: return launch_rows<__half>(p, n_sm, st);
        case 2: return launch_rows<__nv_bfloat16>(p, n_sm, st);
        default: return launch_rows<float>(p, n_sm, st);
    }
}

int launch_token_grad(const TokenGradParams &p, cudaStream_t st) {
    switch (p.dtype) {
        case 1: return launch_grad<__half>(p, st);
        case 2: return launch_grad<__nv_bfloat16>(p, st);
        default: return launch_grad<float>(p, st);
    }
}

}  // namespace moe
