// Host build of the entry points of the vocabulary's operators and the 16-bit dense
// layers (csrc/operators.cu) next to the others', over the same stand-in for the CUDA
// runtime; kernel launches write a line.
#include "api_host.cpp"

#define fail operators_fail  // (both files have one of their own)
#include "operators.cu"
#undef fail

namespace moe {
int launch_token_logprobs(const TokenParams &p, int, cudaStream_t st) {
    return launch("token_logprobs", st, p.logits, p.logp, p.n_tokens);
}
int launch_token_grad(const TokenGradParams &p, cudaStream_t st) {
    return launch("token_grad", st, p.logits, p.dlogits, p.n_tokens);
}
int dense_steps(const DenseProduct &p) { return (p.K + 127) / 128 * p.n_pairs; }
DensePlan dense_plan(const DenseProduct *, int n, int, int) { return DensePlan{256, 128, 1, 1, 1, n * 100.0}; }
int launch_dense_few(const DenseFew &p, int, cudaStream_t st) { return launch("dense_few", st, p.x, p.o.out, p.n_tokens); }
int launch_dense_split(const DenseSplit &p, cudaStream_t st) {
    return launch("dense_split", st, p.src, p.parts, p.n_parts);
}
int launch_dense_gemm(DenseGemm &g, const DensePlan &, int, int, cudaStream_t st) {
    return launch("dense_gemm", st, g.p[0].o.out, g.n_products > 1 ? g.p[1].o.out : nullptr, g.n_products);
}
int launch_dense_join(const float *parts, int shares, size_t, void *out, int, int, cudaStream_t st) {
    return launch("dense_join", st, parts, out, shares);
}
}  // namespace moe
