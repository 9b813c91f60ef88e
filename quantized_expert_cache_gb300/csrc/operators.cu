// Entry points of the vocabulary's operators and the 16-bit dense layers: checks of
// their arguments and their launches.  See moe_cache.h for the contract of each.
#include "../../include/moe_cache.h"
#include "kernels.h"
#include "operands.h"

#include <cmath>

namespace {

using moe::apart;
using moe::Span;
using moe::whole;

int fail(moe_ctx *ctx, int code, const std::string &msg) { return moe::op_fail(ctx, code, msg); }

size_t size_of(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == MOE_F32 || dtype == MOE_F16 || dtype == MOE_BF16; }

// The context's device while a call launches; the caller's own again after it.
struct OnDevice {
    int before = -1;
    explicit OnDevice(int device) {
        int now = device;
        if (cudaGetDevice(&now) == cudaSuccess && now != device && cudaSetDevice(device) == cudaSuccess) before = now;
    }
    ~OnDevice() {
        if (before >= 0) cudaSetDevice(before);
    }
};

int launched(moe_ctx *ctx, const char *what, int rc) {
    if (!rc) return MOE_OK;
    return fail(ctx, MOE_ERR_CUDA, std::string(what) + " launch: " + cudaGetErrorString((cudaError_t)rc));
}

// What both calls over the vocabulary ask of their sizes.
int token_sizes(moe_ctx *ctx, const char *what, int dtype, int n_tokens, int vocab, float scale) {
    if (!known(dtype)) return fail(ctx, MOE_ERR_ARG, std::string(what) + ": dtype must be MOE_F32, MOE_F16 or MOE_BF16");
    if (n_tokens < 0 || vocab < 1 || vocab > moe::kTokenMaxVocab || !(scale > 0.0f) || !std::isfinite(scale))
        return fail(ctx, MOE_ERR_ARG,
                    std::string(what) + ": need n_tokens >= 0, 1 <= vocab <= 2^30, a positive finite scale");
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_token_logprobs(moe_ctx *ctx, const void *d_logits, int dtype, const int32_t *d_targets, int n_tokens,
                       int vocab, float scale, int n_top, float *d_logp, float *d_entropy, int32_t *d_top_idx,
                       float *d_top_logp, float *d_stats, void *stream) {
    if (!ctx) return fail(nullptr, MOE_ERR_ARG, "null ctx");
    const int rc = token_sizes(ctx, "token_logprobs", dtype, n_tokens, vocab, scale);
    if (rc) return rc;
    if (n_top < 0 || n_top > moe::kTokenMaxTop || n_top > vocab)
        return fail(ctx, MOE_ERR_ARG, "token_logprobs: need 0 <= n_top <= min(32, vocab)");
    if (n_tokens == 0) return MOE_OK;
    if (!d_logits || (n_top > 0 && (!d_top_idx || !d_top_logp)) || (d_logp && !d_targets) ||
        (!d_logp && !d_entropy && !d_stats && n_top == 0))
        return fail(ctx, MOE_ERR_ARG, "token_logprobs: null pointer (d_logp needs d_targets; at least one output)");
    if (!whole({d_logits}, size_of(dtype)) || !whole({d_targets, d_logp, d_entropy, d_stats}, 4) ||
        (n_top > 0 && !whole({d_top_idx, d_top_logp}, 4)))
        return fail(ctx, MOE_ERR_ARG, "token_logprobs: a pointer is not aligned to its elements");
    const size_t t = (size_t)n_tokens, row = t * 4, top = row * n_top;
    if (!apart({{d_logits, t * vocab * size_of(dtype)}, {d_targets, row}},
               {{d_logp, row}, {d_entropy, row}, {top ? d_top_idx : nullptr, top}, {top ? d_top_logp : nullptr, top},
                {d_stats, 2 * row}}))
        return fail(ctx, MOE_ERR_ARG, "token_logprobs: an output meets another buffer");
    const moe::OpContext c = moe::op_context(ctx);
    moe::TokenParams p{};
    p.logits = d_logits;
    p.targets = d_targets;
    p.logp = d_logp;
    p.entropy = d_entropy;
    p.top_idx = d_top_idx;
    p.top_logp = d_top_logp;
    p.stats = d_stats;
    p.error = c.error;
    p.dtype = dtype;
    p.n_tokens = n_tokens;
    p.vocab = vocab;
    p.n_top = n_top;
    p.scale = scale;
    const OnDevice on(c.device);
    return launched(ctx, "token_logprobs",
                    moe::launch_token_logprobs(p, c.n_sm, stream ? (cudaStream_t)stream : c.stream));
}

int moe_token_logprobs_grad(moe_ctx *ctx, const void *d_logits, int dtype, const int32_t *d_targets, int n_tokens,
                            int vocab, float scale, const float *d_stats, const float *d_entropy,
                            const float *d_g_logp, const float *d_g_entropy, void *d_dlogits, void *stream) {
    if (!ctx) return fail(nullptr, MOE_ERR_ARG, "null ctx");
    const int rc = token_sizes(ctx, "token_logprobs_grad", dtype, n_tokens, vocab, scale);
    if (rc) return rc;
    if (n_tokens == 0) return MOE_OK;
    if (!d_logits || !d_stats || !d_dlogits || (!d_g_logp && !d_g_entropy) || (d_g_logp && !d_targets) ||
        (d_g_entropy && !d_entropy))
        return fail(ctx, MOE_ERR_ARG,
                    "token_logprobs_grad: null pointer (d_g_logp needs d_targets, d_g_entropy needs d_entropy)");
    if (!whole({d_logits, d_dlogits}, size_of(dtype)) ||
        !whole({d_targets, d_stats, d_entropy, d_g_logp, d_g_entropy}, 4))
        return fail(ctx, MOE_ERR_ARG, "token_logprobs_grad: a pointer is not aligned to its elements");
    const size_t t = (size_t)n_tokens, row = t * 4, n = t * vocab * size_of(dtype);
    if (!apart({{d_dlogits == d_logits ? nullptr : d_logits, n}, {d_targets, row}, {d_stats, 2 * row},
                {d_entropy, row}, {d_g_logp, row}, {d_g_entropy, row}},
               {{d_dlogits, n}}))
        return fail(ctx, MOE_ERR_ARG, "token_logprobs_grad: d_dlogits meets another buffer (it may be d_logits)");
    const moe::OpContext c = moe::op_context(ctx);
    moe::TokenGradParams p{};
    p.logits = d_logits;
    p.targets = d_targets;
    p.stats = d_stats;
    p.entropy = d_entropy;
    p.g_logp = d_g_logp;
    p.g_entropy = d_g_entropy;
    p.dlogits = d_dlogits;
    p.error = c.error;
    p.dtype = dtype;
    p.n_tokens = n_tokens;
    p.vocab = vocab;
    p.scale = scale;
    const OnDevice on(c.device);
    return launched(ctx, "token_logprobs_grad",
                    moe::launch_token_grad(p, stream ? (cudaStream_t)stream : c.stream));
}

}  // extern "C"
