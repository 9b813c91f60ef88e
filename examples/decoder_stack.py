"""A small stack of MoE layers with an output head, token by token: the
library's operators as a decoder uses them together.

    for each layer:  residual sum and RMS norm (fp32 rows for the experts, int8
                     codes for the product), the router as a 4-bit linear layer
                     on the codes, the routed experts
    at the end:      the last norm, the output head as a 4-bit linear layer,
                     the promotion pass of the expert cache
    to answer:       the log probabilities of the tokens taken, the entropies and
                     the likeliest alternatives

and, for a router that is tuned on the way, the balance and z loss of every
layer with the gradient of its logits, and the picks of every expert: the
routing-frequency table that seeds a context's pools.

    python examples/decoder_stack.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_expert_cache_gb300 as qec  # noqa: E402
import synth  # noqa: E402

EPS = 1e-6


class DecoderStack:
    """Random weights of seeded streams; every buffer a step needs is kept."""

    def __init__(self, hidden=256, ffn=512, experts=8, top_k=2, layers=2, vocab=1000, max_tokens=16, slots=4, seed=0):
        self.H, self.E, self.k, self.L, self.V, self.M = hidden, experts, top_k, layers, vocab, max_tokens
        self.wl = synth.Workload("stack", hidden, experts, top_k, ffn, layers, seed=seed)
        self.ctx = qec.moe_layer_init(hidden, ffn, experts, top_k, layers, slots, max_tokens,
                                      stream=torch.cuda.current_stream().cuda_stream)
        self.tensors, self.routers, self.router_w = {}, [], []
        for layer in range(layers):
            for kind in range(3):
                rows, cols = self.wl.tensor_shapes[kind]
                t = self.tensors[layer, kind] = self.wl.expert_tensor(layer, kind)
                qec.register_expert_tensor(self.ctx, layer, kind, t, rows, cols, slots, None, slots)
            w = synth.q4_blocks(synth.key(seed, 100, layer), experts * hidden // 32).reshape(experts, -1, 18)
            self.router_w.append(w)
            self.routers.append(qec.moe_linear_register(self.ctx, w, qec.FMT_Q4_0, experts, hidden))
        self.head_w = synth.q4_blocks(synth.key(seed, 101), vocab * hidden // 32).reshape(vocab, -1, 18)
        self.head = qec.moe_linear_register(self.ctx, self.head_w, qec.FMT_Q4_0, vocab, hidden)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.norms = [1 + 0.1 * torch.randn(hidden, generator=g, device="cuda") for _ in range(layers + 1)]
        empty = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        m, n = max_tokens, layers + 1
        self.stream_rows = [empty(m, hidden) for _ in range(n)]
        self.y = [empty(m, hidden) for _ in range(n)]
        self.q = [empty(m, hidden, dtype=torch.int8) for _ in range(n)]
        self.d = [empty(m, hidden // 32, dtype=torch.float16) for _ in range(n)]
        self.logits = [empty(m, experts) for _ in range(layers)]
        self.idx = [empty(m, top_k, dtype=torch.int32) for _ in range(layers)]
        self.w = [empty(m, top_k) for _ in range(layers)]
        self.out = [empty(m, hidden) for _ in range(layers)]
        self.head_logits = empty(m, vocab)

    def close(self):
        torch.cuda.synchronize()
        qec.moe_destroy(self.ctx)
        self.ctx = None

    def _norm(self, i, x, res, n):
        qec.moe_rms_norm(self.ctx, x, res, self.norms[i], n, self.H, EPS, self.stream_rows[i], self.y[i], self.q[i],
                         self.d[i])

    def step(self, x):
        """fp32 rows [n][hidden] of this step's tokens -> logits [n][vocab]."""
        n = x.shape[0]
        for layer in range(self.L):
            if layer == 0:
                self._norm(0, x, None, n)
            else:
                self._norm(layer, self.out[layer - 1], self.stream_rows[layer - 1], n)
            qec.moe_linear_forward(self.ctx, self.routers[layer], None, n, self.logits[layer], q=self.q[layer],
                                   d=self.d[layer])
            qec.moe_ffn_forward_routed(self.ctx, layer, self.y[layer], self.logits[layer], n, self.idx[layer],
                                       self.w[layer], self.out[layer])
        self._norm(self.L, self.out[-1], self.stream_rows[self.L - 1], n)
        qec.moe_linear_forward(self.ctx, self.head, None, n, self.head_logits, q=self.q[self.L], d=self.d[self.L])
        qec.cache_step(self.ctx, n)
        return self.head_logits[:n]

    def answer(self, tokens, n_top):
        """Of the last step's logits, for int32 tokens [n]: (log probabilities [n], entropies [n], the n_top likeliest
        tokens [n][n_top], their log probabilities)."""
        n = tokens.shape[0]
        made = [torch.empty(n, device="cuda"), torch.empty(n, device="cuda"),
                torch.empty(n, n_top, dtype=torch.int32, device="cuda"), torch.empty(n, n_top, device="cuda")]
        logp, entropy, idx, alternatives = made
        qec.moe_token_logprobs(self.ctx, self.head_logits, tokens, n, self.V, logp, entropy, n_top, idx, alternatives)
        return made

    def router_losses(self, n, mask=None, balance=0.01, z=0.001):
        """Of the last step: per layer (losses [2], picks [E], the logits' gradient [n][E])."""
        made = []
        for layer in range(self.L):
            loss = torch.empty(2, device="cuda")
            counts = torch.empty(self.E, dtype=torch.int32, device="cuda")
            dz = torch.empty(n, self.E, device="cuda")
            qec.moe_router_loss(self.ctx, self.logits[layer], self.idx[layer], mask, None, n, self.E, self.k, balance,
                                z, loss, counts, dz)
            made.append((loss, counts, dz))
        return made


def main():
    stack = DecoderStack()
    g = torch.Generator(device="cuda").manual_seed(1)
    embed = torch.randn(stack.V, stack.H, generator=g, device="cuda")
    tokens = torch.randint(0, stack.V, (4,), generator=g, device="cuda")
    picks = torch.zeros(stack.L, stack.E, dtype=torch.int64, device="cuda")
    for step in range(8):
        logits = stack.step(embed[tokens])
        made = stack.router_losses(tokens.numel())
        for layer, (_, counts, _) in enumerate(made):
            picks[layer] += counts
        tokens = logits.argmax(1)
        logp, _, _, _ = stack.answer(tokens.to(torch.int32), 4)
        print(f"step {step}: tokens {tokens.tolist()}, log probabilities "
              + " ".join(f"{float(v):.3f}" for v in logp) + ", balance loss "
              + " ".join(f"{float(loss[0]):.5f}" for loss, _, _ in made))
    for layer in range(stack.L):
        order = np.argsort(-picks[layer].cpu().numpy(), kind="stable")
        print(f"layer {layer}: seed order {order.tolist()}, cache {qec.moe_stats(stack.ctx)['hits']} hits")
    stack.close()


if __name__ == "__main__":
    main()
