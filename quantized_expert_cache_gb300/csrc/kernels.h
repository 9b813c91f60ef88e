// Internal interface between the C-ABI runtime (moe_cache.cu) and the
// kernels.  Not part of the public ABI.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <cuda.h>
#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {

struct PlanParams {
    const float *x;       // [T][H] (quantized when quantize_x)
    int8_t *xq;           // [T][H]
    BlockScale *xds;      // [T][H/32]
    const int32_t *idx;   // [T][k]
    int32_t *n_uniq;      // [1]
    int32_t *uniq_e;      // [min(T*k, E)]
    int32_t *uniq_off;    // [min(T*k, E) + 1]
    int32_t *assign;      // [T*k]: assignment ids grouped by expert
    int *error;           // [1]: bit 0 = expert id out of range
    int T, k, E, H, quantize_x;
    // expert shard: ids are global in [0, E_route); this context holds
    // [e_base, e_base + E) (local id = id - e_base); assignments to other
    // experts are left out of every used-expert list (placed after them in
    // assign) and contribute nothing
    int e_base, E_route;
};

struct GemvParams {
    CacheView cv;
    int tid_gate, tid_up, tid_down;
    int n_tokens, k, H, F;
    const int8_t *xq;
    const BlockScale *xds;
    const int32_t *n_uniq, *uniq_e, *uniq_off, *assign;
    int8_t *hq;           // [T*k][F]
    BlockScale *hds;      // [T*k][F/32]
    float *o;             // [T*k][H]
    unsigned *counters;   // [H / rows per down item], zero between launches
    const float *w;       // [T][k]
    float *y;             // [T][H]
    int8_t *xq_out;       // fused path: [T][H] copy of the quantized x
    BlockScale *xds_out;  // fused path: [T][H/32]
    int fmt;              // weight format of the mat-vec kernels (kFmtQ4 / kFmtQ8)
    const int32_t *idx;   // [T][k] global expert ids (the combine skips experts of other shards)
    int e_base;           // first expert of this shard (local id = global id - e_base)
};

// Fused small-batch layer (cooperative launch).
struct FusedParams {
    GemvParams g;
    const float *x;          // [T][H]
    const int32_t *idx;      // [T][k] (when logits is null)
    const float *logits;     // [T][n_route]: route in-kernel (top-k + softmax) when not null
    int n_route;             // experts of the whole layer (logit columns; global id range)
    int32_t *idx_out;        // routed: [T][k] written by CTA 0
    float *w_out;            // routed: [T][k] written by CTA 0
    int renorm;
    int pdl;                 // launched with programmatic stream serialization
    unsigned *done_gu;       // [E]: published gate/up row blocks per expert (row-block mode: per
                             // used-expert index), zero between launches
    unsigned *exit_count;    // [1]
    int *error;
    // Row-block down mode (rb_rows > 0): a down item is rb_rows rows of H for
    // every used expert, so it sums y itself; done_gu is then indexed by the
    // used-expert index.  pre_off: shared-memory offset of the down prefetch
    // area.
    int rb_rows;
    int pre_off;
    // One routed token in row-block mode (fused_t1_ok): shared-memory offset
    // of the layer's gate, up and down table rows (0: the general prologue).
    int tbl_off;
    // 1: the last assignment of the token is the layer's shared expert (table
    // column E - 1 of the launch's rows, weight 1), which the single-token
    // path starts at kernel entry; 0: routed experts only
    int n_shared;
    // Lookahead (one routed token, early-start path): predict the next
    // layer's picks as the top-k of pr_b + pr_w . x and prefetch their
    // pool-resident weights into L2 (pr_w null: off).
    const __nv_bfloat16 *pr_w;    // [E][H] router of the next layer
    const float *pr_b;            // [E] its bias
    const uint64_t *pr_tbl;       // [3][E] the next layer's gate, up and down table rows
    float *pr_z;                  // [E] scratch: predicted logits
    unsigned *pr_count;           // [1] predicted logits written (zero between launches)
    unsigned *pr_flag;            // [1] the prediction is out (zero between launches)
    int32_t *pr_set;              // [k] this launch's prediction for the next layer
    const int32_t *pr_mine;       // [k] the previous layer's prediction for this one (or null)
    unsigned long long *pr_stats; // [2] predicted picks, of them actually picked
    size_t pr_blob;               // bytes of one expert tensor blob
};

// One grouped GEMM launch (gate/up with SwiGLU + h quantization, or down).
struct GemmParams {
    const int32_t *n_uniq, *uniq_e, *uniq_off, *tile_off, *assign;
    const uint2 *tile_rec;      // per tile: (u | row tile << 16, token tile | valid columns << 16)
    const uint64_t *tbl[2];     // expert tables of the A operands (gate, up) or (down, -)
    const float *a_scaleT;      // [K/32][A_pad]: block scales of the sorted activation rows
    int rows, K;                // weight rows (output features) and reduction length
    int A, A_pad, k, F_out;
    __half *hq16;               // gate/up: [A_pad][F] sorted h codes as fp16
    float *hdT;                 // gate/up: [F/32][A_pad] sorted h scales
    int8_t *hq;                 // gate/up: [A][F] h codes by assignment
    BlockScale *hds;            // gate/up: [A][F/32] by assignment
    float *o;                   // down: [A][H] by assignment
    int *error;                 // bit set when a bounded wait expires
};

struct TilingParams {
    CacheView cv;
    const int32_t *n_uniq, *uniq_e, *uniq_off;
    int32_t *tile_off_gu, *tile_off_dn;
    uint2 *rec_gu, *rec_dn;
    int cap_gu, cap_dn;
    int tid0, n_tokens, rt_gu, bn_gu, rt_dn, bn_dn;
};

struct PrefillLaunch {
    TilingParams tiling;
    GemmParams gu, dn;
    CUtensorMap tm_x, tm_h;     // sorted fp16 activations / h codes, 128-B swizzle
    const int8_t *xq;
    const BlockScale *xds;
    __half *xs16;
    float *xdT;
    const float *w;
    float *y;
    int T, k, H, n_sm;
    const int32_t *idx;         // [T][k] global expert ids (the combine skips other shards' experts)
    int e_base, E;              // this shard's experts: global ids [e_base, e_base + E)
};

// Staging of a prefill layer's cold expert tensors into lent pool slots.
struct StageParams {
    const uint64_t *tbl;      // [n_tensors][E]
    uint64_t *etbl;           // [3][E]: effective table rows of the layer
    const int32_t *n_uniq, *uniq_e;
    uint64_t *jobs;           // [2 * n_slots]: (source, destination) per staged blob
    int *n_jobs;
    uint64_t slot_base, slot_stride;
    int n_slots, tid0, E;
};

// One table / slot / stamp write of the promotion pass.
struct Update {
    uint32_t what;   // 0: tbl[index] = value; 1: slot[index] = value; 2: stamps[index] = value
    uint32_t index;
    uint64_t value;
};

// Residual addition, RMS norm and int8 output (kernels_norm.cu).
struct NormParams {
    const void *x, *res;        // [n_tokens][width] of dtype; res may be null
    void *sum;                  // [n_tokens][width] of dtype, or null
    const float *weight;        // [width]
    float *y;                   // [n_tokens][width], or null
    int8_t *q;                  // [n_tokens][width], or null (width % 32 == 0)
    __half *d;                  // [n_tokens][width / 32] with q
    int dtype;                  // 0 fp32, 1 binary16, 2 bfloat16
    int n_tokens, width;
    float eps;
};

// Router balance and z loss with the logits' gradient (kernels_router.cu).
constexpr int kRouterParts = 1024;  // CTAs of the loss kernel at most
struct RouterParams {
    const float *logits;        // [T][E]
    const int32_t *idx;         // [T][k]
    const uint8_t *mask;        // [T] or null: 0 leaves the token out
    const float *gw;            // [T][k] or null: gradient of the routing weights
    float *loss;                // [2]
    int32_t *counts;            // [E]
    float *dlogits;             // [T][E] or null
    int32_t *ws_count;          // [E + 1]: picks and unmasked tokens, zero between calls
    unsigned *ticket;           // [2], zero between launches
    float *ws_part;             // [kRouterParts][2]
    int *error;                 // bit 0: an id out of range
    int T, E, k, renorm;
    float balance, zcoef;
};

// Log probabilities of tokens and their gradient (kernels_token.cu).
constexpr int kTokenMaxTop = 32, kTokenMaxVocab = 1 << 30;
constexpr int kErrorToken = 128;    // error bit: a target id past the vocabulary
struct TokenParams {
    const void *logits;         // [T][vocab] of dtype
    const int32_t *targets;     // [T] or null; below 0: none
    float *logp, *entropy;      // [T] or null
    int32_t *top_idx;           // [T][n_top]
    float *top_logp;            // [T][n_top]
    float *stats;               // [T][2] or null: largest logit, log of the sum relative to it
    int *error;                 // kErrorToken
    int dtype, n_tokens, vocab, n_top;
    float scale;
};
struct TokenGradParams {
    const void *logits;         // [T][vocab] of dtype
    const int32_t *targets;     // [T] or null
    const float *stats;         // [T][2]
    const float *entropy;       // [T] with g_entropy
    const float *g_logp, *g_entropy;  // [T] or null
    void *dlogits;              // [T][vocab] of dtype, may be logits
    int *error;
    int dtype, n_tokens, vocab;
    float scale;
};

// 16-bit dense layers (kernels_dense.cu, kernels_dense_gemm.cu).
constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2;
constexpr int kErrorDense = 256;    // error bit: a bounded wait expired
// Output [columns][ld], element (m, n) at n * ld + m, of dtype (0 fp32, 1 binary16, 2 bfloat16).
struct DenseOut {
    void *out;
    const float *bias;          // [ld] by m, or null
    const void *res;            // as out, added at the end, or null
    void *pre;                  // as out, the sums before the activation, or null
    int dtype, act, ld;
};
// Few tokens: y = act(x W^T + bias) + res, warps to rows of W.  us there and on the tensor
// cores at 2, 3 and 4 tokens (bf16 rows, fp32 result): 512 x 2048 2.0, 2.3, 2.7 and 5.5;
// 512 x 8192 4.0, 4.3, 5.1 and 7.7; 2048 x 2048 3.8, 4.1, 5.0 and 6.7; 1000 x 8192 5.9, 6.5,
// 8.7 and 8.4; 2880 x 2880 7.2, 8.5, 8.3 and 8.2; 8192 x 2048 7.6, 10.4, 10.0 and 9.9; 8192 x
// 8192 25.5, 35.4, 33.1 and 26.2; 65536 x 2048 44.3, 52.9, 56.1 and 43.8.
inline bool dense_takes_few(int n_tokens, int rows, int cols) {
    return n_tokens <= 2 || (n_tokens <= 4 && (long long)rows * cols <= 1 << 22);
}
// Up to so many tokens the parts of fp32 rows are columns of one product, which reads
// the weights once; above they are further steps of it.
constexpr int kDenseFold = 64;
// A binary16 gradient times a slope (up to 1.13) passes binary16's range where the gradient is
// near its end: the parts of it are held by half, the finished sums doubled.  The second part
// is held 2^12 larger than that: 2^-11 of the first and less, it would sink into binary16's
// subnormal numbers.  (At most 16 of a first part up to 37009, and so 2^16: cut to 65504, that
// is 2^-22 of the whole.)
constexpr float kDenseHold = 0.5f, kDenseLowScale = 4096.0f, kDenseMost16 = 65504.0f;
struct DenseFew {
    const void *x, *w;          // [n_tokens][cols], [rows][cols]
    int x_dtype, w_dtype, n_tokens, rows, cols;
    DenseOut o;                 // ld = rows
};
// An operand in 16-bit parts whose sum it is, and the sums of its columns.
struct DenseSplit {
    const void *src;            // [n_tokens][cols] of dtype
    const void *pre;            // as src: multiplied by the activation's slope there, or null
    int dtype, act, n_tokens, cols;
    void *parts;                // [n_parts][n_tokens][ld], or by_row: [n_tokens][n_parts][ld]; or null
    int n_parts, ld, by_row;
    float *sums;                // [cols] or null, through
    float *ws_sums;             // [dense_sum_blocks(n_tokens)][cols]
    int finish;                 // 1: sums are finished too; 0: the products' launch does
    int beside;                 // 1: runs beside the launch before it (of the same call), and ends after it
};
// Tokens of a block of column sums, the blocks, and a bound of them that does not fall as
// the tokens rise.
inline int dense_block_tokens(int n_tokens) { return n_tokens <= 2048 ? 16 : ((n_tokens + 127) / 128 + 7) / 8 * 8; }
inline int dense_sum_blocks(int n_tokens) {
    const int t = dense_block_tokens(n_tokens);
    return (n_tokens + t - 1) / t;
}
inline int dense_most_blocks(int n_tokens) { return n_tokens < 2048 ? (n_tokens + 15) / 16 : 128; }
// One product D[m][n] = sum over pairs of parts and over k of A[m][k] B[n][k].
struct DenseProduct {
    CUtensorMap tm_a, tm_b;     // [part][outer][inner], boxes of 64 x 128 (B with k inner: x box rows)
    int M, N, K;
    int a_mn, b_mn;             // 1: stored [k][m] or [k][n]; 0: [m][k], [n][k]
    int bf16;                   // operands: 1 bfloat16, 0 binary16
    int fold;                   // 1: N counts columns of B, four to a token, whose sum is the token's
    int n_pairs;
    unsigned pairs;             // 4 bits each, the first lowest: part of A | part of B << 2
    int m_tiles, n_tiles;
    float low_scale, scale;     // of the sums of all pairs but the last; of all sums
    DenseOut o;                 // ld = M
    // K shares of a tile, each an own tile whose fp32 sums go to o.out + share * M * N
    // (joined by launch_dense_join); up to most_shares of them
    int shares, most_shares;
};
struct DenseGemm {
    DenseProduct p[2];          // two: the one of more steps a tile first
    int n_products, splits;
    int second[2];              // tiles of the second product for workers with one more of the first, and for the others
    int *error;
    // column sums to finish on the side (sums null: none): [sum_blocks][sum_cols]
    const float *sum_parts;
    float *sums;
    int sum_blocks, sum_cols;
};
int dense_steps(const DenseProduct &p);  // of a tile
// Tile columns, rows of B in one box, whether two CTAs share a tile, K splits over a
// cluster, K shares of the first product, an estimate of its clocks.
struct DensePlan {
    int bn, box, pair, splits, shares;
    double clocks;
};
// out[i] = the sum of `shares` arrays of n fp32 numbers, of dtype.
int launch_dense_join(const float *parts, int shares, size_t n, void *out, int dtype, int n_sm, cudaStream_t st);
DensePlan dense_plan(const DenseProduct *p, int n_products, int device, int n_sm);
int launch_dense_few(const DenseFew &p, int n_sm, cudaStream_t st);
int launch_dense_split(const DenseSplit &p, cudaStream_t st);
int launch_dense_gemm(DenseGemm &g, const DensePlan &plan, int device, int n_sm, cudaStream_t st);

// Dense layer with 4-bit weights (kernels_linear.cu).
constexpr int kLinearMaxCols = 65536, kLinearMaxRows = 1 << 26;
constexpr int kLinearSmem = 200 * 1024;        // dynamic shared memory of a CTA
// Whether a batch goes to the tensor cores: from 5 tokens on, and 3 or 4 of more
// than 2048 columns (what the dp4a kernel's CTAs all stage and read from shared
// memory).  3 tokens, us there and on the tensor cores: 512 x 512 2.4 and 6.6, 512
// x 2048 5.5 and 6.7, 8192 x 2048 8.7 and 10.4, 65536 x 2048 26.3 and 45.0, 2880 x
// 2880 9.7 and 8.0, 8192 x 8192 32.9 and 26.8.  Columns alone misjudge many rows
// of a few more columns: 65536 x 4096 50.6 and 82.8.
inline bool linear_takes_gemm(int n_tokens, int cols) { return n_tokens > 4 || (n_tokens > 2 && cols > 2048); }
struct LinearParams {
    const uint8_t *w;           // the weights, layout of linear.cuh
    const float *x;             // [n_tokens][cols], or null and the codes below
    const int8_t *q;            // [n_tokens][cols]
    const __half *d;            // [n_tokens][cols / 32]
    float *y;                   // [n_tokens][rows]
    int fmt, rows, cols, n_tokens;
    // batches: the activations' two binary16 halves [max_tokens][cols] and their
    // token scales
    __half *ws_hi, *ws_lo;
    float *ws_scale;
    int *error;                 // a bit set when a bounded wait expires
};
struct LinearGemm {
    CUtensorMap tm_hi, tm_lo;   // the halves, 128-B swizzle, boxes of linear_gemm_box() tokens
    LinearParams p;
};

int launch_rms_norm(const NormParams &p, cudaStream_t st);
int launch_router_loss(const RouterParams &p, int n_sm, cudaStream_t st);
int launch_token_logprobs(const TokenParams &p, int n_sm, cudaStream_t st);
int launch_token_grad(const TokenGradParams &p, cudaStream_t st);
size_t linear_weight_bytes(int fmt, int rows, int cols);
int launch_linear_repack(const uint8_t *src, uint8_t *dst, int fmt, int rows, int cols, int n_sm, cudaStream_t st);
int launch_linear_max(uint8_t *w, int fmt, int rows, int cols, unsigned *out, int n_sm, cudaStream_t st);
int launch_linear(const LinearParams &p, int n_sm, cudaStream_t st);
int linear_gemm_box();
int linear_gemm_configure();
int launch_linear_gemm(const LinearGemm &g, int n_sm, cudaStream_t st);
int launch_topk(const float *logits, int T, int E, int k, int renorm, int32_t *idx, float *w, cudaStream_t st);
int launch_quantize(const float *x, int n_blocks, int8_t *q, BlockScale *ds, int n_sm, cudaStream_t st);
int launch_plan(const PlanParams &p, cudaStream_t st);
int launch_gemv(const GemvParams &p, int grid_gu, int grid_dn, cudaStream_t st, cudaEvent_t const *ev = nullptr);
int down_rows_per_item(int F);
int launch_block_dots(const uint8_t *blob, int fmt, int rows, int nb, int row0, int n_rows, const int8_t *qa,
                      int32_t *out, cudaStream_t st);
int launch_stream_read(const void *src, size_t bytes, uint32_t *sink, int n_sm, cudaStream_t st);
size_t fused_smem_bytes(int H, int F);
int fused_configure(int F, size_t smem, int *blocks_per_sm);
int fused_rb_rows(int H, int F, int T, int k, int E);
size_t fused_rb_smem(int H, int F, int T, int k, int E, int rows, int *pre_off);
bool fused_t1_ok(int E, int k);
int fused_configure_rb(int F, size_t smem, int *blocks_per_sm);
int fused_configure_t1_fmt(int F, int fmt, size_t smem, int *blocks_per_sm);
int launch_fused(const FusedParams &p, int grid, size_t smem, cudaStream_t st, cudaEvent_t const *ev);
int launch_prefill(const PrefillLaunch &L, cudaStream_t st, cudaEvent_t const *ev = nullptr);
int launch_stage(const StageParams &p, size_t blob_bytes, int n_sm, cudaStream_t st);
int launch_prefetch_table(const uint64_t *tbl_rows, const int32_t *map, const void *buf, int cap, size_t stride,
                          int E, uint64_t *etbl, cudaStream_t st);
int gemm_configure();
int gemm_bn(bool dual);
int gemm_rows_per_tile(bool dual);
int launch_step_finish(const Update *u, int n, uint64_t *tbl, int32_t *slot, uint32_t *stamps, uint32_t *clock,
                       uint32_t new_clock, uint32_t *clear_a, int n_a, uint32_t *clear_b, int n_b, cudaStream_t st);
int launch_count_assign(const int32_t *idx, int n, int E, int e_base, uint32_t *cnt, cudaStream_t st);
int launch_busy(unsigned long long ns, cudaStream_t st);
int launch_shared_assign(const int32_t *idx, const float *w, int T, int k, int e_shared, int32_t *idx_a, float *w_a,
                         int *error, cudaStream_t st);

}  // namespace moe
