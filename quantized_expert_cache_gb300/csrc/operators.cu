// Entry points of the vocabulary's operators and the 16-bit dense layers: checks of
// their arguments and their launches.  See moe_cache.h for the contract of each.
#include "../../include/moe_cache.h"
#include "kernels.h"
#include "operands.h"

#include <cudaTypedefs.h>

#include <algorithm>
#include <utility>

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
    // (the kernels' scale / ln 2 is finite: the largest logit is 0 times it)
    if (n_tokens < 0 || vocab < 1 || vocab > moe::kTokenMaxVocab || !(scale > 0.0f) || scale > 0x1p127f)
        return fail(ctx, MOE_ERR_ARG,
                    std::string(what) + ": need n_tokens >= 0, 1 <= vocab <= 2^30, a positive scale up to 2^127");
    return MOE_OK;
}

// ---- dense layers ------------------------------------------------------------
constexpr long long kDenseMost = 1ll << 38;  // elements of a matrix
constexpr int kDenseSide = 1 << 26;          // rows, columns or tokens

size_t round_up(size_t n, size_t to) { return (n + to - 1) / to * to; }

int dense_sizes(moe_ctx *ctx, const char *what, int x_dtype, int w_dtype, int y_dtype, int act, int n_tokens, int rows,
                int cols) {
    const std::string name = what;
    if (w_dtype != MOE_F16 && w_dtype != MOE_BF16)
        return fail(ctx, MOE_ERR_ARG, name + ": w_dtype must be MOE_F16 or MOE_BF16");
    if (x_dtype != w_dtype && !(x_dtype == MOE_F32 && w_dtype == MOE_BF16))
        return fail(ctx, MOE_ERR_ARG, name + ": x_dtype must be w_dtype, or MOE_F32 with MOE_BF16 weights");
    if (y_dtype != MOE_F32 && y_dtype != w_dtype)
        return fail(ctx, MOE_ERR_ARG, name + ": y_dtype must be MOE_F32 or w_dtype");
    if (act != MOE_ACT_NONE && act != MOE_ACT_SILU && act != MOE_ACT_GELU)
        return fail(ctx, MOE_ERR_ARG, name + ": unknown activation");
    if (n_tokens < 0 || n_tokens > kDenseSide || rows < 1 || rows > kDenseSide || cols < 8 || cols % 8 ||
        cols > kDenseSide || (long long)rows * cols > kDenseMost || (long long)n_tokens * rows > kDenseMost ||
        (long long)n_tokens * cols > kDenseMost)
        return fail(ctx, MOE_ERR_ARG, name + ": need 0 <= n_tokens, 1 <= rows, cols % 8 == 0 (each up to 2^26, matrices "
                                             "up to 2^38 elements)");
    return MOE_OK;
}

// Parts of an operand of the tensor cores (kernels_dense.cu says why).
int row_parts(int x_dtype, bool f32_result) { return x_dtype != MOE_F32 ? 1 : f32_result ? 3 : 2; }
int gradient_parts(int dtype, bool slope, bool f32_result) {
    if (dtype != MOE_F32 && !slope) return 1;
    return f32_result && dtype != MOE_F16 ? 3 : 2;
}
// K shares of the weights' gradient: what 32 MB of sums hold.
int weight_shares(int rows, int cols) { return (int)std::min<size_t>(8, ((size_t)32 << 20) / ((size_t)rows * cols * 4)); }

// Regions of a call's workspace.
struct DenseSpace {
    size_t x_parts = 0, z_parts = 0, sums = 0, shares = 0, bytes = 0;  // offsets
};
DenseSpace dense_space(bool backward, int x_dtype, int y_dtype, int act, int n_tokens, int rows, int cols) {
    DenseSpace s;
    const auto take = [&](size_t n) {
        const size_t at = s.bytes;
        s.bytes += round_up(n, 256);
        return at;
    };
    const size_t t = (size_t)n_tokens;
    if (!backward) {
        if (x_dtype == MOE_F32 && !moe::dense_takes_few(n_tokens, rows, cols)) s.x_parts = take(t * cols * 3 * 2);
        return s;
    }
    if (x_dtype == MOE_F32) s.x_parts = take(t * cols * 3 * 2);
    s.z_parts = take(t * round_up(rows, 8) * gradient_parts(y_dtype, act != MOE_ACT_NONE, true) * 2);
    s.sums = take((size_t)moe::dense_most_blocks(n_tokens) * rows * 4);
    if (weight_shares(rows, cols) > 1) s.shares = take((size_t)weight_shares(rows, cols) * rows * cols * 4);
    return s;
}

// [part][outer][inner] in boxes of 64 x box_outer; fold: [outer][part][inner], a box has four
// parts (those past the last are zero) of a fourth as many rows.
int encode_map(moe_ctx *ctx, CUtensorMap *tm, const void *base, bool bf16, size_t inner, size_t outer, size_t ld,
               int parts, uint32_t box_outer, bool fold) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? (PFN_cuTensorMapEncodeTiled_v12000)fn : nullptr;
    }();
    if (!encode) return fail(ctx, MOE_ERR_CUDA, "cuTensorMapEncodeTiled entry point not found");
    const cuuint64_t n_parts = (cuuint64_t)parts, middle = fold ? n_parts : outer, last = fold ? outer : n_parts;
    const cuuint64_t dims[3] = {inner, middle, last}, strides[2] = {ld * 2, middle * ld * 2};
    const cuuint32_t box[3] = {64, fold ? 4 : box_outer, fold ? box_outer / 4 : 1}, one[3] = {1, 1, 1};
    const CUresult r = encode(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                              (void *)base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MOE_OK : fail(ctx, MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed");
}

// A matrix [outer][inner] (rows of ld elements, in parts) as an operand.
struct DenseMatrix {
    const void *base;
    size_t inner, outer, ld;
    int parts;
};

// The pairs of parts a product takes, those up to `most` of the places in all, the largest
// products last.
void dense_pairs(moe::DenseProduct &p, int a_parts, int b_parts, int most) {
    p.n_pairs = 0;
    p.pairs = 0;
    for (int sum = most; sum >= 0; --sum)
        for (int a = 0; a <= sum; ++a)
            if (a < a_parts && sum - a < b_parts)
                p.pairs |= (unsigned)(a | (sum - a) << 2) << (4 * p.n_pairs++);
}

int dense_launch(moe_ctx *ctx, moe::DenseGemm &g, const DenseMatrix *a, const DenseMatrix *b, const moe::DensePlan &plan,
                 float *sums, const moe::OpContext &c, cudaStream_t st, const char *what) {
    g.splits = plan.splits;
    g.error = c.error;
    for (int i = 0; i < g.n_products; ++i) g.p[i].shares = 1;
    const moe::DenseOut joined = g.p[0].o;
    if (plan.shares > 1) {
        g.p[0].shares = plan.shares;
        g.p[0].o.out = sums;
        g.p[0].o.dtype = MOE_F32;
    }
    for (int i = 0; i < g.n_products; ++i) {
        moe::DenseProduct &p = g.p[i];
        const int rc = encode_map(ctx, &p.tm_a, a[i].base, p.bf16, a[i].inner, a[i].outer, a[i].ld, a[i].parts,
                                  128, false);
        if (rc) return rc;
        const int rd = encode_map(ctx, &p.tm_b, b[i].base, p.bf16, b[i].inner, b[i].outer, b[i].ld, b[i].parts,
                                  p.b_mn ? 128 : (uint32_t)plan.box, p.fold);
        if (rd) return rd;
    }
    const int rc = launched(ctx, what, moe::launch_dense_gemm(g, plan, c.device, c.n_sm, st));
    if (rc || plan.shares == 1) return rc;
    return launched(ctx, what, moe::launch_dense_join(sums, plan.shares, (size_t)g.p[0].M * g.p[0].N, joined.out,
                                                      joined.dtype, c.n_sm, st));
}

// The products of a call (their pairs of parts set), two of them in one launch (their
// tiles fill the SMs together) or in two (each with its own tiles and K splits), as the
// plans have it.
int dense_products(moe_ctx *ctx, moe::DenseGemm &g, DenseMatrix *a, DenseMatrix *b, float *sums,
                   const moe::OpContext &c, cudaStream_t st, const char *what) {
    if (g.n_products == 2 && moe::dense_steps(g.p[0]) < moe::dense_steps(g.p[1])) {
        std::swap(g.p[0], g.p[1]);
        std::swap(a[0], a[1]);
        std::swap(b[0], b[1]);
    }
    const moe::DensePlan all = moe::dense_plan(g.p, g.n_products, c.device, c.n_sm);
    if (g.n_products == 1) return dense_launch(ctx, g, a, b, all, sums, c, st, what);
    const moe::DensePlan one = moe::dense_plan(g.p, 1, c.device, c.n_sm),
                         two = moe::dense_plan(g.p + 1, 1, c.device, c.n_sm);
    constexpr double kLaunch = 5000;  // clocks
    if (all.clocks <= one.clocks + two.clocks + kLaunch) return dense_launch(ctx, g, a, b, all, sums, c, st, what);
    g.n_products = 1;
    const int rc = dense_launch(ctx, g, a, b, one, sums, c, st, what);
    if (rc) return rc;
    g.p[0] = g.p[1];
    g.sums = nullptr;
    return dense_launch(ctx, g, a + 1, b + 1, two, sums, c, st, what);
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

int moe_dense_workspace(moe_ctx *ctx, int x_dtype, int w_dtype, int y_dtype, int act, int n_tokens, int rows, int cols,
                        size_t *forward_bytes, size_t *backward_bytes) {
    if (!ctx) return fail(nullptr, MOE_ERR_ARG, "null ctx");
    const int rc = dense_sizes(ctx, "dense_workspace", x_dtype, w_dtype, y_dtype, act, n_tokens, rows, cols);
    if (rc) return rc;
    if (forward_bytes) *forward_bytes = dense_space(false, x_dtype, y_dtype, act, n_tokens, rows, cols).bytes;
    if (backward_bytes) *backward_bytes = dense_space(true, x_dtype, y_dtype, act, n_tokens, rows, cols).bytes;
    return MOE_OK;
}

int moe_dense_forward(moe_ctx *ctx, const void *d_x, int x_dtype, const void *d_w, int w_dtype, const float *d_bias,
                      int act, const void *d_res, int n_tokens, int rows, int cols, void *d_y, int y_dtype,
                      void *d_pre, void *d_ws, size_t ws_bytes, void *stream) {
    if (!ctx) return fail(nullptr, MOE_ERR_ARG, "null ctx");
    const int rc = dense_sizes(ctx, "dense", x_dtype, w_dtype, y_dtype, act, n_tokens, rows, cols);
    if (rc) return rc;
    if (n_tokens == 0) return MOE_OK;
    if (!d_x || !d_w || !d_y) return fail(ctx, MOE_ERR_ARG, "dense: null pointer");
    const DenseSpace space = dense_space(false, x_dtype, y_dtype, act, n_tokens, rows, cols);
    if (space.bytes && (!d_ws || ws_bytes < space.bytes))
        return fail(ctx, MOE_ERR_ARG, "dense: need a workspace of " + std::to_string(space.bytes) + " bytes");
    void *ws = space.bytes ? d_ws : nullptr;
    if (!whole({d_x, d_w, ws}, 16) || !whole({d_bias}, 4) || !whole({d_res, d_y, d_pre}, size_of(y_dtype)))
        return fail(ctx, MOE_ERR_ARG,
                    "dense: d_x, d_w and the workspace must be 16-byte aligned, the others to their elements");
    const size_t t = (size_t)n_tokens, xn = t * cols * size_of(x_dtype), wn = (size_t)rows * cols * 2,
                 yn = t * rows * size_of(y_dtype);
    if (!apart({{d_x, xn}, {d_w, wn}, {d_bias, (size_t)rows * 4}, {d_res == d_y ? nullptr : d_res, yn}},
               {{d_y, yn}, {d_pre, yn}, {ws, space.bytes}}))
        return fail(ctx, MOE_ERR_ARG, "dense: an output or the workspace meets another buffer (d_y may be d_res)");
    const moe::OpContext c = moe::op_context(ctx);
    const cudaStream_t st = stream ? (cudaStream_t)stream : c.stream;
    const OnDevice on(c.device);
    const moe::DenseOut out{d_y, d_bias, d_res, d_pre, y_dtype, act, rows};
    if (moe::dense_takes_few(n_tokens, rows, cols)) {
        const moe::DenseFew f{d_x, d_w, x_dtype, w_dtype, n_tokens, rows, cols, out};
        return launched(ctx, "dense", moe::launch_dense_few(f, c.n_sm, st));
    }
    DenseMatrix x{d_x, (size_t)cols, t, (size_t)cols, row_parts(x_dtype, y_dtype == MOE_F32)};
    if (x_dtype == MOE_F32) {
        moe::DenseSplit s{};
        s.src = d_x;
        s.dtype = x_dtype;
        s.n_tokens = n_tokens;
        s.cols = s.ld = cols;
        s.parts = (uint8_t *)ws + space.x_parts;
        s.n_parts = x.parts;
        s.by_row = n_tokens <= moe::kDenseFold;
        const int r = launched(ctx, "dense", moe::launch_dense_split(s, st));
        if (r) return r;
        x.base = s.parts;
    }
    DenseMatrix w{d_w, (size_t)cols, (size_t)rows, (size_t)cols, 1};
    moe::DenseGemm g{};
    g.n_products = 1;
    g.p[0].M = rows;
    g.p[0].N = n_tokens;
    g.p[0].K = cols;
    g.p[0].bf16 = w_dtype == MOE_BF16;
    g.p[0].low_scale = g.p[0].scale = 1.0f;
    g.p[0].o = out;
    if (x.parts > 1 && n_tokens <= moe::kDenseFold) {
        g.p[0].fold = 1;
        g.p[0].N = 4 * n_tokens;
    }
    dense_pairs(g.p[0], 1, g.p[0].fold ? 1 : x.parts, x.parts - 1);
    return dense_products(ctx, g, &w, &x, nullptr, c, st, "dense");
}

int moe_dense_backward(moe_ctx *ctx, const void *d_x, int x_dtype, const void *d_w, int w_dtype, const void *d_dy,
                       int y_dtype, const void *d_pre, int act, int n_tokens, int rows, int cols, void *d_dx,
                       void *d_dw, int dw_dtype, float *d_db, void *d_ws, size_t ws_bytes, void *stream) {
    if (!ctx) return fail(nullptr, MOE_ERR_ARG, "null ctx");
    const int rc = dense_sizes(ctx, "dense_backward", x_dtype, w_dtype, y_dtype, act, n_tokens, rows, cols);
    if (rc) return rc;
    if (w_dtype == MOE_F16 && y_dtype == MOE_F32)
        return fail(ctx, MOE_ERR_ARG, "dense_backward: fp32 gradients go with MOE_BF16 weights (binary16 has not their range)");
    if (d_dw && dw_dtype != MOE_F32 && dw_dtype != w_dtype)
        return fail(ctx, MOE_ERR_ARG, "dense_backward: dw_dtype must be MOE_F32 or w_dtype");
    if (!d_dx && !d_dw && !d_db) return fail(ctx, MOE_ERR_ARG, "dense_backward: no output");
    if (!whole({d_dx}, size_of(x_dtype)) || !whole({d_dw}, size_of(dw_dtype)) || !whole({d_db}, 4))
        return fail(ctx, MOE_ERR_ARG, "dense_backward: a pointer is not aligned to its elements");
    const moe::OpContext c = moe::op_context(ctx);
    const cudaStream_t st = stream ? (cudaStream_t)stream : c.stream;
    const size_t t = (size_t)n_tokens, xn = t * cols * size_of(x_dtype), wn = (size_t)rows * cols,
                 yn = t * rows * size_of(y_dtype), dwn = wn * size_of(dw_dtype), dbn = (size_t)rows * 4;
    // (also where no token has anything written to d_dx or the workspace)
    if (!apart({{d_dx ? d_w : nullptr, wn * 2}}, {{d_dw, dwn}, {d_db, dbn}}))
        return fail(ctx, MOE_ERR_ARG, "dense_backward: an output meets another buffer");
    const OnDevice on(c.device);
    if (n_tokens == 0) {
        // sums over no tokens
        cudaError_t e = d_dw ? cudaMemsetAsync(d_dw, 0, dwn, st) : cudaSuccess;
        if (e == cudaSuccess && d_db) e = cudaMemsetAsync(d_db, 0, dbn, st);
        return launched(ctx, "dense_backward", (int)e);
    }
    const bool slope = act != MOE_ACT_NONE;
    if (!d_dy || (slope && !d_pre) || (d_dx && !d_w) || (d_dw && !d_x))
        return fail(ctx, MOE_ERR_ARG,
                    "dense_backward: null pointer (d_dx needs d_w, d_dw needs d_x, an activation needs d_pre)");
    const DenseSpace space = dense_space(true, x_dtype, y_dtype, act, n_tokens, rows, cols);
    if (!d_ws || ws_bytes < space.bytes)
        return fail(ctx, MOE_ERR_ARG, "dense_backward: need a workspace of " + std::to_string(space.bytes) + " bytes");
    const void *pre = slope ? d_pre : nullptr, *x = d_dw ? d_x : nullptr, *w = d_dx ? d_w : nullptr;
    if (!whole({x, w, d_ws}, 16) || !whole({d_dy, pre}, size_of(y_dtype)))
        return fail(ctx, MOE_ERR_ARG,
                    "dense_backward: d_x, d_w and d_ws must be 16-byte aligned, the others to their elements");
    if (!apart({{x, xn}, {w, wn * 2}, {d_dy, yn}, {pre, yn}},
               {{d_dx, xn}, {d_dw, dwn}, {d_db, dbn}, {d_ws, space.bytes}}))
        return fail(ctx, MOE_ERR_ARG, "dense_backward: an output or the workspace meets another buffer");
    uint8_t *ws = (uint8_t *)d_ws;
    const bool f32_result = (d_dx && x_dtype == MOE_F32) || (d_dw && dw_dtype == MOE_F32);
    // dz, as it is if it is 16-bit and its rows are aligned
    const bool product = d_dx || d_dw;
    DenseMatrix dz{d_dy, (size_t)rows, t, (size_t)rows, gradient_parts(y_dtype, slope, f32_result)};
    const bool direct = !slope && y_dtype != MOE_F32 && rows % 8 == 0 && whole({d_dy}, 16);
    moe::DenseGemm g{};
    moe::DenseSplit s{};
    // dz goes first where the products need it; else its sums alone go last, beside the
    // products' tail (4096^3 bf16: 8 us less)
    const bool first = product && !direct;
    if (d_db || first) {
        s.src = d_dy;
        s.pre = pre;
        s.dtype = y_dtype;
        s.act = act;
        s.n_tokens = n_tokens;
        s.cols = rows;
        s.ld = (int)round_up(rows, 8);
        if (product && !direct) {
            s.parts = ws + space.z_parts;
            s.n_parts = dz.parts;
            dz.base = s.parts;
            dz.ld = s.ld;
        }
        s.sums = d_db;
        s.ws_sums = (float *)(ws + space.sums);
        s.finish = !first;
        if (d_db && first) {
            g.sum_parts = s.ws_sums;
            g.sums = d_db;
            g.sum_blocks = moe::dense_sum_blocks(n_tokens);
            g.sum_cols = rows;
        }
        if (first || !product) {
            const int r = launched(ctx, "dense_backward", moe::launch_dense_split(s, st));
            if (r || !product) return r;
        }
    }
    DenseMatrix xs{d_x, (size_t)cols, t, (size_t)cols, 1};
    if (d_dw && x_dtype == MOE_F32) {
        moe::DenseSplit q{};
        q.src = d_x;
        q.dtype = x_dtype;
        q.n_tokens = n_tokens;
        q.cols = q.ld = cols;
        q.parts = ws + space.x_parts;
        q.n_parts = xs.parts = row_parts(x_dtype, dw_dtype == MOE_F32);
        q.beside = first;
        const int r = launched(ctx, "dense_backward", moe::launch_dense_split(q, st));
        if (r) return r;
        xs.base = q.parts;
    }
    DenseMatrix a[2], b[2];
    if (d_dw) {
        moe::DenseProduct &p = g.p[g.n_products];
        p.M = cols;
        p.N = rows;
        p.K = n_tokens;
        p.a_mn = p.b_mn = 1;
        p.o.out = d_dw;
        p.o.dtype = dw_dtype;
        p.most_shares = weight_shares(rows, cols);
        a[g.n_products] = xs;
        b[g.n_products++] = dz;
    }
    if (d_dx) {
        moe::DenseProduct &p = g.p[g.n_products];
        p.M = cols;
        p.N = n_tokens;
        p.K = rows;
        p.a_mn = 1;
        p.o.out = d_dx;
        p.o.dtype = x_dtype;
        a[g.n_products] = DenseMatrix{d_w, (size_t)cols, (size_t)rows, (size_t)cols, 1};
        b[g.n_products++] = dz;
    }
    for (int i = 0; i < g.n_products; ++i) {
        g.p[i].bf16 = w_dtype == MOE_BF16;
        g.p[i].low_scale = w_dtype == MOE_F16 ? 1.0f / moe::kDenseLowScale : 1.0f;
        g.p[i].scale = w_dtype == MOE_F16 && slope ? 1.0f / moe::kDenseHold : 1.0f;
        g.p[i].o.ld = cols;
        dense_pairs(g.p[i], a[i].parts, b[i].parts, g.p[i].o.dtype == MOE_F32 ? 2 : 1);
    }
    const int r = dense_products(ctx, g, a, b, (float *)(ws + space.shares), c, st, "dense_backward");
    if (r || first || !d_db) return r;
    s.beside = 1;
    return launched(ctx, "dense_backward", moe::launch_dense_split(s, st));
}

}  // extern "C"
