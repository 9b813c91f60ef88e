// Balance and z loss of a router, the picks of each expert, and the gradient
// of both (and of the routing weights) with respect to the logits.
//
// Over the n unmasked tokens t, with p_t = softmax(z_t), lse_t = logsumexp(z_t)
// and c_e the picks of expert e:
//   f_e = c_e / (n k)
//   L_bal = a E sum_e f_e mean_t p_te = (a E / n) sum_t (f . p_t)
//   L_z = b mean_t lse_t^2
//   dz_te = p_te (a E (f_e - f . p_t) + 2 b lse_t) / n   (f is a constant)
//         + w_tj (g_tj - sum_i g_ti w_ti) at e = idx_tj  (w: softmax over the
//           picks; with weights read off the softmax over all E instead,
//           p_te (sum_j [idx_tj = e] g_tj - sum_j g_tj p_t,idx_tj))
// The loss needs only the scalars f . p_t and lse_t that the gradient needs
// too, so the logits are read once and no E-wide sum over tokens is kept.
// Counts are integers (their atomics commute exactly); the loss is summed
// in an order that only the grid size sets: results do not vary from run to run.
//
// Bound: 8 tokens (one launch, 3.3 us) by latency; 4096 x 512 with all three
// gradients 10.3 to 10.7 us against 2.5 of HBM's rate, padded 12288 x 512 18.3 to
// 18.6 against 7.5: two dependent launches, then a row's chain of loads and warp
// reductions with 32 warps a SM to hide it.  (Profiled with a cold cache, the
// padded case's counting kernel takes 6 us, the loss kernel 20; it keeps DRAM at 14%
// of its rate and waits most often for loads.  What does not need the counts is not
// yet done before their wait.)
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr size_t kCountInLoss = 4096;
constexpr float kNegInf = -__builtin_inff();

// exp(x) for x <= 0 as 2^(x log2 e) by the special-function unit: 2 ulp and
// |x| 2^-24 of the result, results below 2^-126 are 0.
__device__ __forceinline__ float exp_neg(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}

// An id outside [0, E) is read as expert 0 and reported, as in the forwards.
__device__ __forceinline__ int checked_id(int e, int E, int *error) {
    if ((unsigned)e >= (unsigned)E) {
        atomicOr(error, 1);
        return 0;
    }
    return e;
}

// Picks first, first + step, ... into hist[E] and, at hist[E], the unmasked
// tokens.  Neighbouring lanes take neighbouring picks, of few tokens, so that a
// warp's atomics seldom meet at a popular expert.  Ends with the CTA
// synchronised.
__device__ __forceinline__ void count_picks(const RouterParams &p, int *hist, int first, int step) {
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const size_t n = (size_t)p.T * p.k;
    constexpr int kBatch = 4;  // loads in flight
    int valid = 0;
    for (size_t i0 = first; i0 < n; i0 += (size_t)kBatch * step) {
        int e[kBatch];
        bool on[kBatch], head[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const size_t i = i0 + (size_t)j * step;
            const size_t t = n <= 0xffffffffu ? (unsigned)i / (unsigned)p.k : i / p.k;
            e[j] = i < n ? p.idx[i] : 0;
            on[j] = i < n && (!p.mask || p.mask[t]);
            head[j] = i == t * p.k;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (on[j]) {
                atomicAdd(&hist[checked_id(e[j], p.E, p.error)], 1);
                valid += head[j];
            }
    }
    valid = __reduce_add_sync(0xffffffffu, valid);
    if ((threadIdx.x & 31) == 0 && valid) atomicAdd(&hist[p.E], valid);
    __syncthreads();
}

// Picks per expert of a long batch: the histogram of each CTA's share, added to
// ws_count, which is zero between calls (the loss kernel leaves it so).
// (With one cluster of 16 CTAs that joined its histograms in shared memory the
// padded 12288 x 512 case took 20.2 us in all, 18.3 with this.)
__global__ void __launch_bounds__(kThreads) router_count_kernel(RouterParams p) {
    extern __shared__ int hist[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    count_picks(p, hist, blockIdx.x * kThreads + threadIdx.x, gridDim.x * kThreads);
    for (int e = threadIdx.x; e <= p.E; e += kThreads)
        if (hist[e]) atomicAdd(&p.ws_count[e], hist[e]);
}

// One warp a row, ITEMS packs of VEC logits a lane.  COUNT: a short batch, every CTA counts all
// picks itself (CTA 0 writes them) and no other kernel runs.
template <int VEC, int ITEMS, bool COUNT>
__global__ void __launch_bounds__(kThreads, VEC * ITEMS <= 16 ? 4 : 1) router_loss_kernel(RouterParams p) {
    extern __shared__ __align__(16) float f[];
    __shared__ float part[2][kThreads / 32];
    const int E = p.E, k = p.k, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    struct alignas(4 * VEC) Pack {
        float v[VEC];
    };
    using LoadT = typename std::conditional<VEC == 4, float4, float>::type;
    const int nv = E / VEC;
    const size_t step = (size_t)gridDim.x * (kThreads / 32);
    size_t t = (size_t)blockIdx.x * (kThreads / 32) + warp;
    // A row's logits, and for lane j < k its pick j with the weight's gradient
    // and logit.  What a row's loads depend on (its mask, its picks) is
    // requested a row ahead (meta), the row itself (rows of up to 16 values a
    // lane) while the one before it is worked on.  All through L2: the first
    // rows are read before this grid's dependency wait, when L1 may still hold
    // an earlier launch's lines.
    constexpr bool kAhead = VEC * ITEMS <= 16;
    struct Meta {
        bool on;
        int e;
        float g;
    };
    struct Row {
        Pack z[ITEMS];
        Meta m;
        float zs;
    };
    auto meta = [&](size_t row) {
        Meta m{row < (size_t)p.T, -1, 0.0f};
        if (!m.on) return m;
        if (p.gw && lane < k) {
            m.e = __ldcg(p.idx + row * k + lane);
            m.g = __ldcg(p.gw + row * k + lane);
        }
        if (p.mask) m.on = __ldcg(p.mask + row) != 0;
        return m;
    };
    auto fetch = [&](Row &r, const Meta &m, size_t row) {
        r.m = m;
        r.zs = 0.0f;
        if (!m.on) return;
        const LoadT *zr = (const LoadT *)(p.logits + row * E);
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int v = lane + 32 * i;
            if (v < nv)
                *(LoadT *)&r.z[i] = __ldcg(zr + v);
            else
#pragma unroll
                for (int j = 0; j < VEC; ++j) r.z[i].v[j] = kNegInf;
        }
        if (p.gw && lane < k) {
            r.m.e = checked_id(m.e, E, p.error);
            r.zs = __ldcg(p.logits + row * E + r.m.e);
        }
    };
    Row cur;
    Meta ahead;
    auto start = [&]() {
        const Meta m = meta(t);
        ahead = meta(t + step);
        fetch(cur, m, t);
    };
    int n_valid;
    if (COUNT) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;");
        start();
        int *hist = (int *)f;
        count_picks(p, hist, threadIdx.x, kThreads);
        n_valid = hist[E];
        const float inv_nk = n_valid > 0 ? 1.0f / ((float)n_valid * (float)k) : 0.0f;
        for (int i = threadIdx.x; i < E; i += kThreads) {
            const int c = hist[i];
            if (blockIdx.x == 0) p.counts[i] = c;
            f[i] = (float)c * inv_nk;
        }
    } else {
        // the counting kernel lets this grid start once its own wait is over,
        // so what earlier work wrote is visible here; its counts are not yet
        start();
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;");
        n_valid = __ldcg(p.ws_count + E);
        const float inv_nk = n_valid > 0 ? 1.0f / ((float)n_valid * (float)k) : 0.0f;
        for (int i = threadIdx.x; i < E; i += kThreads) {
            const int c = __ldcg(p.ws_count + i);
            if (blockIdx.x == 0) p.counts[i] = c;
            f[i] = (float)c * inv_nk;
        }
    }
    __syncthreads();
    const float inv_n = n_valid > 0 ? 1.0f / (float)n_valid : 0.0f;
    const float cb = p.balance * (float)E * inv_n, cz = 2.0f * p.zcoef * inv_n;
    float bal = 0.0f, zz = 0.0f;
    // One row: its loss terms and its gradient.
    auto work = [&](Row &r, size_t t) {
        Pack(&z)[ITEMS] = r.z;
        const bool on = r.m.on;
        const int e = r.m.e;
        const float g = r.m.g, zs = r.zs;
        Pack *dr = p.dlogits ? (Pack *)(p.dlogits + t * E) : nullptr;
        float top = kNegInf;
        bool empty = !on;
        if (on) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) top = fmaxf(top, z[i].v[j]);
            top = warp_max(top);
            if (top == kNegInf) {
                // every logit -inf: no expert left.  (A row of NaN has no
                // maximum either, but stays NaN.)
                bool nan = false;
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) nan |= z[i].v[j] != z[i].v[j];
                empty = !__any_sync(0xffffffffu, nan);
            }
        }
        if (empty) {
            // masked, or no expert left: nothing to add, a zero gradient
            if (dr) {
                for (int v = lane; v < nv; v += 32) dr[v] = Pack{};
            }
            return;
        }
        float tot = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int v = lane + 32 * i;
            if (v < nv) {
                const Pack fe = *((const Pack *)f + v);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    z[i].v[j] = exp_neg(z[i].v[j] - top);
                    tot += z[i].v[j];
                    dot = fmaf(z[i].v[j], fe.v[j], dot);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            tot += __shfl_xor_sync(0xffffffffu, tot, o);
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        const float inv = __frcp_rn(tot);
        dot *= inv;
        const float lse = top + logf(tot);
        bal += dot;
        zz = fmaf(lse, lse, zz);
        if (!dr) return;
        // gradient of the routing weights
        float own = 0.0f, all = 0.0f;
        if (p.gw) {
            if (p.renorm) {
                const float ts = warp_max(lane < k ? zs : kNegInf);
                float w = lane < k && ts != kNegInf ? exp_neg(zs - ts) : 0.0f;
                float sw = w, swg = w * g;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    sw += __shfl_xor_sync(0xffffffffu, sw, o);
                    swg += __shfl_xor_sync(0xffffffffu, swg, o);
                }
                const float is = sw != 0.0f ? __frcp_rn(sw) : 0.0f;
                w *= is;
                own = w * (g - swg * is);
            } else {
                own = lane < k ? g * (exp_neg(zs - top) * inv) : 0.0f;
                all = warp_sum_f(own);
            }
        }
        // dz = e^(z - top) (ci f + bi)
        const float ci = cb * inv, bi = (cz * lse - cb * dot - all) * inv;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int v = lane + 32 * i;
            if (v < nv) {
                const Pack fe = *((const Pack *)f + v);
                Pack o;
#pragma unroll
                for (int j = 0; j < VEC; ++j) o.v[j] = z[i].v[j] * fmaf(ci, fe.v[j], bi);
                dr[v] = o;
            }
        }
        if (p.gw) {
            // the picks' elements are written again with their own term (the
            // same element from every lane that holds it)
            const unsigned same = __match_any_sync(0xffffffffu, lane < k ? e : -1 - lane);
            float add = own;
            if (__any_sync(0xffffffffu, same & (same - 1))) {
                // an id given twice (route_topk writes none)
                add = 0.0f;
                for (int j = 0; j < k; ++j) {
                    const float gj = __shfl_sync(0xffffffffu, own, j);
                    if (same >> j & 1) add += gj;
                }
            }
            __syncwarp();
            if (lane < k) p.dlogits[t * E + e] = fmaf(exp_neg(zs - top), fmaf(ci, f[e], bi), add);
        }
    };
    // (two buffers in turn: the unrolled loop copies no row)
    Row next;
    auto turn = [&](Row &now, Row &then) {
        const Meta m = ahead;
        const size_t row = t;
        t += step;
        const bool more = t < (size_t)p.T;
        if (more) ahead = meta(t + step);
        if (kAhead && more) fetch(then, m, t);
        work(now, row);
        if (!kAhead && more) fetch(now, m, t);
        return more;
    };
    if (t < (size_t)p.T) {
        if constexpr (kAhead)
            while (turn(cur, next) && turn(next, cur)) {
            }
        else
            while (turn(cur, cur)) {
            }
    }
    if (lane == 0) {
        part[0][warp] = bal;
        part[1][warp] = zz;
    }
    __syncthreads();
    // the CTA's parts, then (the last CTA) all CTAs': warp 0 the balance parts,
    // warp 1 the z parts, in an order that only the grid size sets
    if (warp >= 2) return;
    float sum = lane < kThreads / 32 ? part[warp][lane] : 0.0f;
    sum = warp_sum_f(sum);
    if (gridDim.x > 1) {
        int last = 0;
        if (lane == 0) {
            p.ws_part[2 * blockIdx.x + warp] = sum;
            __threadfence();
            last = atomicAdd(p.ticket + warp, 1u) == gridDim.x - 1;
            __threadfence();
        }
        if (!__shfl_sync(0xffffffffu, last, 0)) return;
        sum = 0.0f;
#pragma unroll 8
        for (unsigned c = lane; c < gridDim.x; c += 32) sum += __ldcg(&p.ws_part[2 * c + warp]);
        sum = warp_sum_f(sum);
    }
    // (every CTA has read the counts)
    if (!COUNT && warp == 0)
        for (int i = lane; i <= E; i += 32) p.ws_count[i] = 0;
    if (lane == 0) {
        const float n = n_valid > 0 ? (float)n_valid : 1.0f;
        p.loss[warp] = (warp ? p.zcoef : p.balance * (float)E) * sum / n;
        p.ticket[warp] = 0;
    }
}

template <typename K>
int launch_pdl(K kernel, unsigned grid, unsigned block, size_t smem, const RouterParams &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
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

template <bool COUNT>
int launch_loss(const RouterParams &p, int n_sm, cudaStream_t st) {
    const size_t rows = kThreads / 32;
    const unsigned g = (unsigned)std::min<size_t>(((size_t)p.T + rows - 1) / rows + (p.T == 0),
                                                  (size_t)std::min(n_sm * 4, kRouterParts));
    const size_t sm = (size_t)(p.E + 1) * 4;
    const auto a16 = [](const void *q) { return ((uintptr_t)q & 15) == 0; };
    if (p.E % 4 == 0 && a16(p.logits) && a16(p.dlogits)) {
        const int nv = p.E / 4;
        if (nv <= 32) return launch_pdl(router_loss_kernel<4, 1, COUNT>, g, kThreads, sm, p, st);
        if (nv <= 64) return launch_pdl(router_loss_kernel<4, 2, COUNT>, g, kThreads, sm, p, st);
        if (nv <= 128) return launch_pdl(router_loss_kernel<4, 4, COUNT>, g, kThreads, sm, p, st);
        if (nv <= 256) return launch_pdl(router_loss_kernel<4, 8, COUNT>, g, kThreads, sm, p, st);
        return launch_pdl(router_loss_kernel<4, 32, COUNT>, g, kThreads, sm, p, st);
    }
    if (p.E <= 64) return launch_pdl(router_loss_kernel<1, 2, COUNT>, g, kThreads, sm, p, st);
    if (p.E <= 256) return launch_pdl(router_loss_kernel<1, 8, COUNT>, g, kThreads, sm, p, st);
    if (p.E <= 512) return launch_pdl(router_loss_kernel<1, 16, COUNT>, g, kThreads, sm, p, st);
    if (p.E <= 1024) return launch_pdl(router_loss_kernel<1, 32, COUNT>, g, kThreads, sm, p, st);
    return launch_pdl(router_loss_kernel<1, 128, COUNT>, g, kThreads, sm, p, st);
}

}  // namespace

int launch_router_loss(const RouterParams &p, int n_sm, cudaStream_t st) {
    // up to kCountInLoss picks every CTA of the loss kernel counts them all
    if ((size_t)p.T * p.k <= kCountInLoss) return launch_loss<true>(p, n_sm, st);
    const size_t ids = (size_t)p.T * p.k;
    const unsigned grid = (unsigned)std::min<size_t>((ids + 2 * kThreads - 1) / (2 * kThreads), (size_t)n_sm);
    int rc = launch_pdl(router_count_kernel, grid, kThreads, (size_t)(p.E + 1) * 4, p, st);
    return rc ? rc : launch_loss<false>(p, n_sm, st);
}

}  // namespace moe
