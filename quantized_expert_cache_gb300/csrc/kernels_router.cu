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
// Counts are integers (their atomics commute exactly); the loss is summed in
// binary64, per-CTA parts in CTA order: results do not vary from run to run.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr float kNegInf = -__builtin_inff();

// An id outside [0, E) is read as expert 0 and reported, as in the forwards.
__device__ __forceinline__ int checked_id(int e, int E, int *error) {
    if ((unsigned)e >= (unsigned)E) {
        atomicOr(error, 1);
        return 0;
    }
    return e;
}

// Picks per expert and unmasked tokens, into counters that are zero between
// launches; the last CTA publishes them and clears the counters.
__global__ void __launch_bounds__(kThreads) router_count_kernel(RouterParams p) {
    extern __shared__ int hist[];
    __shared__ int last;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int E = p.E, k = p.k;
    for (int e = threadIdx.x; e <= E; e += kThreads) hist[e] = 0;
    __syncthreads();
    const size_t n = (size_t)p.T * k;
    for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (size_t)gridDim.x * kThreads) {
        const size_t t = i / k;
        if (p.mask && !p.mask[t]) continue;
        atomicAdd(&hist[checked_id(p.idx[i], E, p.error)], 1);
        if (i == t * k) atomicAdd(&hist[E], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kThreads)
        if (hist[e]) atomicAdd(&p.ws_count[e], hist[e]);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    for (int e = threadIdx.x; e <= E; e += kThreads) {
        const int c = __ldcg(&p.ws_count[e]);
        p.ws_count[e] = 0;
        if (e < E)
            p.counts[e] = c;
        else
            *p.n_valid = c;
    }
    if (threadIdx.x == 0) *p.ticket = 0;
}

// One warp a row, ITEMS packs of VEC logits a lane.
template <int VEC, int ITEMS>
__global__ void __launch_bounds__(kThreads) router_loss_kernel(RouterParams p) {
    extern __shared__ float f[];
    __shared__ double part[2][kThreads / 32];
    __shared__ int last;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int E = p.E, k = p.k, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n_valid = __ldcg(p.n_valid);
    const float inv_n = n_valid > 0 ? 1.0f / (float)n_valid : 0.0f, inv_nk = inv_n / (float)k;
    for (int e = threadIdx.x; e < E; e += kThreads) f[e] = (float)__ldcg(&p.counts[e]) * inv_nk;
    __syncthreads();
    const float cb = p.balance * (float)E * inv_n, cz = 2.0f * p.zcoef * inv_n;
    double bal = 0.0, zz = 0.0;
    struct alignas(4 * VEC) Pack {
        float v[VEC];
    };
    const int nv = E / VEC;
    for (size_t t = (size_t)blockIdx.x * (kThreads / 32) + warp; t < (size_t)p.T;
         t += (size_t)gridDim.x * (kThreads / 32)) {
        const Pack *zr = (const Pack *)(p.logits + t * E);
        Pack *dr = p.dlogits ? (Pack *)(p.dlogits + t * E) : nullptr;
        const bool on = !p.mask || p.mask[t];
        Pack z[ITEMS];
        float top = kNegInf;
        if (on) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const int v = lane + 32 * i;
                if (v < nv)
                    z[i] = zr[v];
                else
#pragma unroll
                    for (int j = 0; j < VEC; ++j) z[i].v[j] = kNegInf;
            }
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) top = fmaxf(top, z[i].v[j]);
            top = warp_max(top);
        }
        bool empty = !on;
        if (on && top == kNegInf) {
            // every logit -inf: no expert left.  (A row of NaN has no maximum
            // either, but stays NaN.)
            bool nan = false;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) nan |= z[i].v[j] != z[i].v[j];
            empty = !__any_sync(0xffffffffu, nan);
        }
        if (empty) {
            // masked, or no expert left: nothing to add, a zero gradient
            if (dr) {
                for (int v = lane; v < nv; v += 32) dr[v] = Pack{};
            }
            continue;
        }
        float tot = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int v = lane + 32 * i;
            if (v < nv) {
                const Pack fe = *((const Pack *)f + v);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    z[i].v[j] = expf(z[i].v[j] - top);
                    tot += z[i].v[j];
                    dot = fmaf(z[i].v[j], fe.v[j], dot);
                }
            }
        }
        tot = warp_sum_f(tot);
        const float inv = 1.0f / tot;
        dot = warp_sum_f(dot) * inv;
        const float lse = top + logf(tot);
        if (lane == 0) {
            bal += dot;
            zz += (double)lse * lse;
        }
        if (!dr) continue;
        // gradient of the routing weights: lane j < k holds pick j
        float g = 0.0f, all = 0.0f, zs = 0.0f;
        int e = -1;
        if (p.gw) {
            if (lane < k) {
                e = checked_id(p.idx[t * k + lane], E, p.error);
                zs = p.logits[t * E + e];
                g = p.gw[t * k + lane];
            }
            if (p.renorm) {
                const float ts = warp_max(lane < k ? zs : kNegInf);
                float w = lane < k && ts != kNegInf ? expf(zs - ts) : 0.0f;
                const float sw = warp_sum_f(w);
                w = sw > 0.0f ? w / sw : 0.0f;
                g = w * (g - warp_sum_f(w * g));
            } else {
                const float ps = lane < k ? expf(zs - top) * inv : 0.0f;
                g *= ps;
                all = warp_sum_f(g);
            }
        }
        const float base = cz * lse - cb * dot - all;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int v = lane + 32 * i;
            if (v < nv) {
                const Pack fe = *((const Pack *)f + v);
                Pack o;
#pragma unroll
                for (int j = 0; j < VEC; ++j) o.v[j] = z[i].v[j] * inv * fmaf(cb, fe.v[j], base);
                dr[v] = o;
            }
        }
        if (p.gw) {
            // the picks' elements are written again with their own term (the
            // same element from every lane that holds it)
            float add = 0.0f;
            for (int j = 0; j < k; ++j) {
                const float gj = __shfl_sync(0xffffffffu, g, j);
                if (__shfl_sync(0xffffffffu, e, j) == e) add += gj;
            }
            __syncwarp();
            if (lane < k) p.dlogits[t * E + e] = expf(zs - top) * inv * fmaf(cb, f[e], base) + add;
        }
    }
    if (lane == 0) {
        part[0][warp] = bal;
        part[1][warp] = zz;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double b = 0.0, z = 0.0;
        for (int w = 0; w < kThreads / 32; ++w) {
            b += part[0][w];
            z += part[1][w];
        }
        p.ws_part[2 * blockIdx.x] = b;
        p.ws_part[2 * blockIdx.x + 1] = z;
        __threadfence();
        last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
        if (last) {
            __threadfence();
            b = z = 0.0;
            for (unsigned c = 0; c < gridDim.x; ++c) {
                b += __ldcg(&p.ws_part[2 * c]);
                z += __ldcg(&p.ws_part[2 * c + 1]);
            }
            const double n = n_valid > 0 ? (double)n_valid : 1.0;
            p.loss[0] = (float)((double)p.balance * E * b / n);
            p.loss[1] = (float)((double)p.zcoef * z / n);
            *p.ticket = 0;
        }
    }
}

template <typename K>
int launch_pdl(K kernel, unsigned grid, size_t smem, const RouterParams &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

int launch_router_loss(const RouterParams &p, int n_sm, cudaStream_t st) {
    const size_t ids = (size_t)p.T * p.k;
    const unsigned gc = (unsigned)std::min<size_t>((ids + kThreads - 1) / kThreads + (ids == 0), (size_t)n_sm);
    int rc = launch_pdl(router_count_kernel, gc, (size_t)(p.E + 1) * 4, p, st);
    if (rc) return rc;
    const unsigned g =
        (unsigned)std::min<size_t>(((size_t)p.T + 7) / 8 + (p.T == 0), (size_t)std::min(n_sm * 4, kRouterParts));
    const size_t sm = (size_t)p.E * 4;
    const auto a16 = [](const void *q) { return ((uintptr_t)q & 15) == 0; };
    if (p.E % 4 == 0 && a16(p.logits) && a16(p.dlogits)) {
        const int nv = p.E / 4;
        if (nv <= 32) return launch_pdl(router_loss_kernel<4, 1>, g, sm, p, st);
        if (nv <= 64) return launch_pdl(router_loss_kernel<4, 2>, g, sm, p, st);
        if (nv <= 128) return launch_pdl(router_loss_kernel<4, 4>, g, sm, p, st);
        if (nv <= 256) return launch_pdl(router_loss_kernel<4, 8>, g, sm, p, st);
        return launch_pdl(router_loss_kernel<4, 32>, g, sm, p, st);
    }
    if (p.E <= 64) return launch_pdl(router_loss_kernel<1, 2>, g, sm, p, st);
    if (p.E <= 256) return launch_pdl(router_loss_kernel<1, 8>, g, sm, p, st);
    if (p.E <= 1024) return launch_pdl(router_loss_kernel<1, 32>, g, sm, p, st);
    return launch_pdl(router_loss_kernel<1, 128>, g, sm, p, st);
}

}  // namespace moe
