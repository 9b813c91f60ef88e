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
// keeps anyway.  A value that n of these reach is a bound below the n-th largest
// element, and units below it hold none of the n; the others, little more than n of
// them, are read again (from L2).  What reaches the bound there, seldom more than a few
// dozen elements, is put in order by counting what comes before each; where it is more
// than kCand, lists of 32 sorted over a warp's lanes take it in and are merged pairwise.
// That is so for ties and masked rows, and for rows of no more units than alternatives,
// which leave no bound: with 32 of them fp32 rows up to 4096 logits and of 8200 to 16384
// (their tiles are four times as large), 16-bit ones up to 8192.  Keys hold the value over
// the inverted index, so order and ties (the lowest index) are one comparison of whole
// numbers, whatever the order of work.
//
// A row takes a cluster of 1 to 8 CTAs.  They write their units' maxima into each other's
// shared memory, their sums and candidates into the first one's: no workspace, any
// stream, one launch.
//
// Bound.  Many rows: HBM; 4096 x 65536 fp32 with 5 alternatives 176 us = 0.90 of a copy
// (158 without: a row's second part stands behind other rows' reads).  bf16 167 = 0.47
// (147 without): issue, 19 instructions an element, which this form takes and the data do
// not ask for.  Gradients: bf16 163 = 0.97, fp32 308 = 1.02.  Few rows: latency; 1 x 65536
// with 8 alternatives 5.6 us (3.8 without), 32 x 100003 bf16 with 20 9.6 (6.3), gradient of
// 33 x 32003 2.4.  Rows that go to the lists: 64 x 2000 fp32 with 20 alternatives 16.7 us
// (6.1 with 8), 32 x 12000 with 32 34; a masked row of 65536 with fewer tokens left than
// alternatives wanted 31.
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

// 16-bit values rounded in pairs: one by one, the conversions share the special-function
// unit with the exponentials.
__device__ __forceinline__ Pack16<float> packed(const float *v, float) { return Pack16<float>{v[0], v[1], v[2], v[3]}; }
__device__ __forceinline__ Pack16<__half> packed(const float *v, __half) {
    Pack16<__half> o;
#pragma unroll
    for (int j = 0; j < 8; j += 2) *(__half2 *)&o.v[j] = __floats2half2_rn(v[j], v[j + 1]);
    return o;
}
__device__ __forceinline__ Pack16<__nv_bfloat16> packed(const float *v, __nv_bfloat16) {
    Pack16<__nv_bfloat16> o;
#pragma unroll
    for (int j = 0; j < 8; j += 2) *(__nv_bfloat162 *)&o.v[j] = __floats2bfloat162_rn(v[j], v[j + 1]);
    return o;
}

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

// A row: `head` elements up to the first 16-byte boundary, `packs` packs of 16 bytes,
// the rest.  Elements outside the packs (fewer than 32) are a lane each.
template <typename T>
struct Row {
    static constexpr int N = 16 / (int)sizeof(T);
    const T *x;
    int head, packs, edge;
    __device__ __forceinline__ Row(const void *logits, size_t row, int vocab)
        : x((const T *)logits + row * (size_t)vocab) {
        head = min(vocab, (int)((16 - ((uintptr_t)x & 15)) % 16 / sizeof(T)));
        packs = (vocab - head) / N;
        edge = vocab - packs * N;
    }
    __device__ __forceinline__ Pack16<T> load(int pack) const { return *(const Pack16<T> *)(x + head + pack * N); }
    // the index of edge element i
    __device__ __forceinline__ int edge_at(int i) const { return i < head ? i : i + packs * N; }
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

// A list of 32 keys over the lanes, largest in lane 0; only the first n_top are wanted.
struct List {
    unsigned long long mine = 0, last = 0;  // last: the n_top-th
    // one candidate a lane (0: none)
    __device__ __forceinline__ void insert(unsigned long long cand, int n_top, int lane) {
        unsigned who = __ballot_sync(0xffffffffu, cand > last);
        while (who) {
            const unsigned long long one = __shfl_sync(0xffffffffu, cand, __ffs(who) - 1);
            who &= who - 1;
            if (one > last) {
                const int at = __popc(__ballot_sync(0xffffffffu, mine > one));
                const unsigned long long up = __shfl_up_sync(0xffffffffu, mine, 1);
                mine = lane < at ? mine : lane == at ? one : up;
                last = __shfl_sync(0xffffffffu, mine, n_top - 1);
            }
        }
    }
};
__device__ __forceinline__ unsigned long long candidate(float x, int index) {
    return (unsigned long long)order_of(x) << 32 | (0xffffffffu - (unsigned)index);
}

constexpr int kCand = 256;     // candidates that are ordered by counting, one a thread
static_assert(kCand <= kThreads && kUnits <= kThreads, "one thread to a unit and to a candidate");

struct TokenShared {
    Sums part[kTokenWarps];        // of the warps
    Sums ctas[kTokenCluster];      // of the CTAs (in the first)
    unsigned unit[kUnits];         // the maxima of the row's units
    unsigned low[kTokenWarps], high[kTokenWarps];  // of the warps' units
    unsigned long long cand[kCand];  // (in the first CTA)
    unsigned long long list[kTokenWarps][kList];
    int flagged[kUnits];
    int n_flagged, n_cand;
    float top, log_sum;            // the row's
    bool none;
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
    const int units = (r.packs + (TILE << shift) - 1) / (TILE << shift);
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
    // Sums of K elements a lane, `high` the largest of the warp's.
    const auto add = [&](const float *x, int K, float high) {
        if (high > a.m) {
            if (a.m != -kInf) lower(a, c * (a.m - high));
            a.m = high;
        }
        // (all -infinity so far: relative to 0 they stay it)
        const float m = a.m == -kInf ? 0.0f : a.m;
        if (high < a.m) {
#pragma unroll
            for (int e = 0; e < K; ++e) {
                const float u = bounded((x[e] - m) * c), f = exp2_neg(u);
                a.s += f;
                a.t = fmaf(f, u, a.t);
            }
        } else {
#pragma unroll
            for (int e = 0; e < K; ++e) {
                const float u = bounded((x[e] - m) * c), f = exp2_neg(u);
                const bool is_max = u == 0.0f;
                a.n += is_max ? 1.0f : 0.0f;
                a.s += is_max ? 0.0f : f;
                a.t = fmaf(f, u, a.t);
            }
        }
    };
    const bool edges = rank == 0 && warp == 0 && r.edge > 0;
    const float x_edge = edges && lane < r.edge ? value<T>(r.x[r.edge_at(lane)]) : -kInf;
    if (edges) add(&x_edge, 1, of_order(__reduce_max_sync(0xffffffffu, order_of(fmaxf(x_edge, -kInf)))));
    const int mine = u0 + warp < u1 ? (u1 - u0 - warp + kTokenWarps - 1) / kTokenWarps : 0;
    const int tiles = mine << shift;
    const auto tile_pack = [&](int i) {
        const int unit = u0 + warp + (i >> shift) * kTokenWarps;
        return ((unit << shift) + (i & ((1 << shift) - 1))) * TILE + lane;
    };
    Pack16<T> none16;
#pragma unroll
    for (int j = 0; j < N; ++j) none16.v[j] = rounded<T>(-kInf);
    const auto tile_load = [&](Pack16<T> *v, int at) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            v[k] = none16;
            if (at + 32 * k < r.packs) v[k] = r.load(at + 32 * k);
        }
    };
    Pack16<T> next[U];
    if (tiles > 0) tile_load(next, tile_pack(0));
    if (threadIdx.x == 0) sh.n_flagged = 0, sh.n_cand = 0;
    if (C > 1)
        cluster.sync();  // (all CTAs have started: their shared memory may be written)
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
        if (i + 1 < tiles) tile_load(next, tile_pack(i + 1));
        const unsigned key = __reduce_max_sync(0xffffffffu, order_of(high));
        top = max(top, key);
        if ((i & ((1 << shift) - 1)) == (1 << shift) - 1) {
            unsigned *unit = &sh.unit[u0 + warp + (i >> shift) * kTokenWarps];
            if (lane < C) *(C > 1 ? cluster.map_shared_rank(unit, lane) : unit) = top;
            top = 0;
        }
        add(x, U * N, of_order(key));
    }
    a.s = warp_sum_f(a.s);
    a.n = warp_sum_f(a.n);
    a.t = warp_sum_f(a.t);
    if (lane == 0) sh.part[warp] = a;
    __syncthreads();
    if (warp == 0) {
        a = joined_lanes<kTokenWarps>(sh.part[lane % kTokenWarps], c);
        if (lane == 0) *(C > 1 ? cluster.map_shared_rank(&sh.ctas[rank], 0) : &sh.ctas[0]) = a;
    }
    if (C > 1)
        cluster.sync();
    else
        __syncthreads();

    // ---- elements that may be among the n largest
    unsigned bound = 0;  // (0: every unit may hold one)
    const unsigned mine_key = (int)threadIdx.x < units ? sh.unit[threadIdx.x] : 0;
    if (p.n_top > 0) {
        if (units > p.n_top) {
            const unsigned least = (int)threadIdx.x < units ? mine_key : 0xffffffffu;
            const unsigned lo = __reduce_min_sync(0xffffffffu, least), hi = __reduce_max_sync(0xffffffffu, mine_key);
            if (lane == 0) sh.low[warp] = lo, sh.high[warp] = hi;
            __syncthreads();
            unsigned from = sh.low[0], to = sh.high[0];
#pragma unroll
            for (int w = 1; w < kTokenWarps; ++w) from = min(from, sh.low[w]), to = max(to, sh.high[w]);
            // the largest value that n_top maxima reach lies in [from, to]; one that a few
            // more reach will do
            for (;;) {
                bound = from;
                if (from == to) break;
                const unsigned middle = to - (to - from) / 2;
                const int reach = __syncthreads_count(mine_key >= middle);
                if (reach >= p.n_top) {
                    bound = from = middle;
                    if (reach <= p.n_top + p.n_top / 2 + 4) break;
                } else {
                    to = middle - 1;
                }
            }
        }
        if ((int)threadIdx.x >= u0 && (int)threadIdx.x < u1 && mine_key >= bound)
            sh.flagged[atomicAdd(&sh.n_flagged, 1)] = threadIdx.x;
        __syncthreads();
        int *n_cand = C > 1 ? cluster.map_shared_rank(&sh.n_cand, 0) : &sh.n_cand;
        unsigned long long *cands = C > 1 ? cluster.map_shared_rank(sh.cand, 0) : sh.cand;
        // A candidate of every lane that has one; false once there are too many.
        const auto offer = [&](bool on, float x, int index) {
            const unsigned who = __ballot_sync(0xffffffffu, on);
            if (!who) return true;
            int at = 0;
            if (lane == 0) at = atomicAdd(n_cand, __popc(who));
            at = __shfl_sync(0xffffffffu, at, 0);
            const int mine_at = at + __popc(who & ((1u << lane) - 1));
            if (on && mine_at < kCand) cands[mine_at] = candidate(x, index);
            return at < kCand;
        };
        bool room = true;
        if (edges)
            room = offer(lane < r.edge && order_of(x_edge) >= bound, x_edge, r.edge_at(lane));
        const int n_flagged = sh.n_flagged;
        for (int f = warp; f < n_flagged && room; f += kTokenWarps) {
            const int first = (sh.flagged[f] << shift) * TILE;
            for (int i = first; i < first + (TILE << shift) && room; i += TILE) {
                Pack16<T> v[U];
                tile_load(v, i + lane);
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int at = i + 32 * k + lane;
                    unsigned high = 0;
#pragma unroll
                    for (int j = 0; j < N; ++j) high = max(high, order_of(value<T>(v[k].v[j])));
                    if (!__any_sync(0xffffffffu, at < r.packs && high >= bound)) continue;
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float x = value<T>(v[k].v[j]);
                        room &= offer(at < r.packs && order_of(x) >= bound, x, r.head + at * N + j);
                    }
                }
            }
        }
        if (C > 1)
            cluster.sync();
        else
            __syncthreads();
    }
    if (rank > 0) return;  // (nothing reads or writes the other CTAs' memory from here on)

    // ---- results
    if (warp == 0) {
        static_assert(kTokenCluster <= kTokenWarps, "one lane to a CTA");
        Sums q = lane % kTokenWarps < C ? sh.ctas[lane % kTokenWarps] : Sums{-kInf, 0.0f, 0.0f, 0.0f};
        q = joined_lanes<kTokenWarps>(q, c);
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
            sh.top = q.m;
            sh.log_sum = log_sum;
            sh.none = none;
        }
    }
    if (p.n_top == 0) return;
    __syncthreads();
    const auto write = [&](int place, unsigned long long key) {
        p.top_idx[row * p.n_top + place] = (int32_t)(0xffffffffu - (unsigned)key);
        p.top_logp[row * p.n_top + place] =
            sh.none ? -kInf : (of_order((unsigned)(key >> 32)) - sh.top) * p.scale - sh.log_sum;
    };
    const int n = sh.n_cand;
    if (n <= kCand) {
        const unsigned long long key = (int)threadIdx.x < n ? sh.cand[threadIdx.x] : 0;
        int before = 0;
        for (int j = 0; j < n; ++j) before += sh.cand[j] > key ? 1 : 0;
        if ((int)threadIdx.x < n && before < p.n_top) write(before, key);
        return;
    }
    // more: all of the row's units that reach the bound, by the first CTA
    if (threadIdx.x == 0) sh.n_flagged = 0;
    __syncthreads();
    if ((int)threadIdx.x < units && mine_key >= bound) sh.flagged[atomicAdd(&sh.n_flagged, 1)] = threadIdx.x;
    __syncthreads();
    List list;
    if (edges) list.insert(lane < r.edge ? candidate(x_edge, r.edge_at(lane)) : 0, p.n_top, lane);
    const int n_flagged = sh.n_flagged;
    for (int f = warp; f < n_flagged; f += kTokenWarps) {
        const int first = (sh.flagged[f] << shift) * TILE;
        for (int i = first; i < first + (TILE << shift); i += TILE) {
            Pack16<T> v[U];
            tile_load(v, i + lane);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                // (a NaN's key is above all others; one past the packs is no candidate)
                unsigned high = 0;
#pragma unroll
                for (int j = 0; j < N; ++j) high = max(high, order_of(value<T>(v[k].v[j])));
                const int at = i + 32 * k + lane, e0 = r.head + at * N;
                // (the best that the pack can hold: a masked row's many equal elements end here)
                const unsigned long long most = (unsigned long long)high << 32 | (0xffffffffu - (unsigned)e0);
                const bool any = at < r.packs && high >= bound && most > list.last;
                if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll 1
                for (int j = 0; j < N; ++j) {
                    float y = 0.0f;
#pragma unroll
                    for (int q = 0; q < N; ++q)
                        if (q == j) y = value<T>(v[k].v[q]);
                    list.insert(any && order_of(y) >= bound ? candidate(y, e0 + j) : 0, p.n_top, lane);
                }
            }
        }
    }
    const unsigned long long best = merge_warps(sh.list, list.mine, warp, lane);
    if (warp == 0 && lane < p.n_top) write(lane, best);
}

// ---- gradient: one read, one write, a row's scalars in every thread --------------
struct GradRow {
    float top, log_sum, scale, by_log, by_one;
    float at_zero;  // the factor without scale
    // -p (by_log log p + by_one): all of a logit's gradient but a target's own term.
    __device__ __forceinline__ float of(float x) const {
        const float lp = fmaf(x - top, scale, -log_sum), p = exp2_neg(lp * kLog2e);
        // (where p is 0, log p or scale may have taken the factor past fp32's range)
        return -p * (p == 0.0f ? at_zero : fmaf(by_log, lp, by_one));
    }
};

// A CTA takes kThreads x kTokenGradPacks packs of a row, all loads of a thread in flight
// together.  Results go where the logits were, to the same thread, when the two buffers
// are one.
template <typename T>
__global__ void __launch_bounds__(kThreads) token_grad_kernel(TokenGradParams p, int chunks, bool same_align) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int N = Pack16<T>::N, PACKS = kTokenGradPacks, SPAN = kThreads * PACKS;
    const size_t row = blockIdx.x / chunks;
    const Row<T> r(p.logits, row, p.vocab);
    T *dx = (T *)p.dlogits + row * (size_t)p.vocab;
    // packs from the boundary at or below the row's first element
    const int before = (int)(((uintptr_t)r.x & 15) / sizeof(T));
    const int pack0 = (int)(blockIdx.x % chunks) * SPAN, e0 = (pack0 + (int)threadIdx.x) * N - before;
    const auto whole = [&](int e) { return same_align && e >= 0 && e + N <= p.vocab; };
    Pack16<T> v[PACKS];
#pragma unroll
    for (int k = 0; k < PACKS; ++k)
        if (whole(e0 + k * kThreads * N)) v[k] = *(const Pack16<T> *)(r.x + e0 + k * kThreads * N);
    int target = p.targets ? p.targets[row] : -1;
    if (target >= p.vocab) {
        if (threadIdx.x == 0) atomicOr(p.error, kErrorToken);
        target = -1;
    }
    GradRow w;
    w.top = p.stats[2 * row];
    w.log_sum = p.stats[2 * row + 1];
    w.scale = p.scale;
    const float g = p.g_logp && target >= 0 ? p.g_logp[row] : 0.0f;
    const float gh = p.g_entropy ? p.g_entropy[row] : 0.0f, h = p.g_entropy ? p.entropy[row] : 0.0f;
    w.by_log = gh * p.scale;
    w.at_zero = fmaf(gh, h, g);
    w.by_one = w.at_zero * p.scale;
    // nothing but -infinity: every p is 0, and so are the gradients
    const bool none = w.top == -kInf && w.log_sum == 0.0f;
    if (none) w.top = w.at_zero = 0.0f;
    // the thread that has the target's pack: g (1 - p) by expm1, so that a likely target's
    // keeps its digits (read before the pack is stored over it)
    const int at = target < 0 ? -1 : (target + before) / N - pack0;
    const bool mine = at >= 0 && at < SPAN && at % kThreads == (int)threadIdx.x;
    float d_target = 0.0f;
    if (mine) {
        const float lp = fmaf(value<T>(r.x[target]) - w.top, p.scale, -w.log_sum);
        d_target = -p.scale * fmaf(exp2_neg(lp * kLog2e) * gh, fmaxf(lp, -150.0f) + h, g * expm1f(lp));
    }
    bool edge = false;
#pragma unroll
    for (int k = 0; k < PACKS; ++k) {
        const int e = e0 + k * kThreads * N;
        if (whole(e)) {
            float d[N];
#pragma unroll
            for (int j = 0; j < N; ++j) d[j] = w.of(value<T>(v[k].v[j]));
            *(Pack16<T> *)(dx + e) = packed(d, T());
        } else {
            edge |= e + N > 0 && e < p.vocab;
        }
    }
    // a row's first and last pack, and rows whose gradients lie otherwise than the logits
    if (edge)
#pragma unroll 1
        for (int k = 0; k < PACKS; ++k) {
            const int e = e0 + k * kThreads * N;
            if (!whole(e))
#pragma unroll 1
                for (int i = max(e, 0); i < min(e + N, p.vocab); ++i) dx[i] = rounded<T>(w.of(value<T>(r.x[i])));
        }
    if (mine && !none) dx[target] = rounded<T>(d_target);
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
    const int packs = p.vocab / N;  // or one less, by the head
    int shift = 0;
    while ((packs + (TILE << shift) - 1) / (TILE << shift) > kUnits) ++shift;
    const int units = std::max(1, (packs + (TILE << shift) - 1) / (TILE << shift));
    // CTAs of a row: as many as keep every warp at a unit, up to four CTAs a SM
    int C = 1;
    while (C < kTokenCluster && (long long)p.n_tokens * C * 2 <= 4ll * n_sm && units >= 2 * C * kTokenWarps) C *= 2;
    auto kernel = token_logprobs_kernel<T, U>;
    return launch(kernel, (size_t)p.n_tokens * C, C, st, p, shift, (units + C - 1) / C);
}

template <typename T>
int launch_rows(const TokenParams &p, int n_sm, cudaStream_t st) {
    // tiles of one pack a lane where 16 elements a lane would make few units to choose
    // from; else 16 (a tile's own work, 60 instructions, to twice the elements: 4096 x
    // 65536 bf16 207 us in tiles of 8)
    constexpr int N = 16 / (int)sizeof(T);
    return p.vocab <= 32 * 64 * N ? launch_logprobs<T, 1>(p, n_sm, st)
                                           : launch_logprobs<T, 16 / N>(p, n_sm, st);
}

template <typename T>
int launch_grad(const TokenGradParams &p, cudaStream_t st) {
    // (64 bytes a thread: 4096 x 65536 bf16 166 us with a cold cache; 32 bytes 269, 128 173)
    constexpr int N = 16 / (int)sizeof(T), PACKS = kTokenGradPacks;
    const int packs = (p.vocab + N - 1) / N + 1, chunks = (packs + kThreads * PACKS - 1) / (kThreads * PACKS);
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
