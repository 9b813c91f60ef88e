"""GPU test of the example stack: every step of a decoder that runs the norm,
the 4-bit linear layers, the routed experts and the router loss together,
each checked from the inputs it was given.

Tolerances are those of the operators' own tests (norm: 46 u, u = 2^-24;
linear: (6 nb + 16) 2^-23 of the sum of |products|) and of the layers' parity
tests (1e-4 + 2e-3 |y|, on the codes the forward used)."""
import os
import sys

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
U = 2.0 ** -24


def q4(w):
    d = w[:, :, :2].copy().view(np.float16).astype(np.float64)
    q = np.concatenate([w[:, :, 2:] & 15, w[:, :, 2:] >> 4], 2).astype(np.float64) - 8
    return (d * q).reshape(w.shape[0], -1)


def f64(t, n):
    return t[:n].cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("n", [1, 2, 7, 16])
def test_stack_steps(n):
    from decoder_stack import EPS, DecoderStack

    s = DecoderStack(slots=8)
    g = torch.Generator(device="cuda").manual_seed(n)
    for step in range(2):
        x = torch.randn(n, s.H, generator=g, device="cuda")
        got = s.step(x)
        losses = s.router_losses(n)
        torch.cuda.synchronize()
        prev = f64(x, n)
        for i in range(s.L + 1):
            sums = prev.astype(np.float32) if i == 0 else (prev.astype(np.float32) + f64(s.stream_rows[i - 1], n).astype(
                np.float32))
            assert np.array_equal(sums, s.stream_rows[i][:n].cpu().numpy())
            v = sums.astype(np.float64)
            ref = v / np.sqrt((v * v).mean(1, keepdims=True) + EPS) * f64(s.norms[i], s.H)
            y = f64(s.y[i], n)
            assert (np.abs(y - ref) <= 46 * U * np.abs(ref) + U * np.abs(v)).all()
            codes = f64(s.q[i], n).reshape(n, -1, 32) * f64(s.d[i], n)[..., None]
            assert (np.abs(codes.reshape(n, -1) - y) <= np.repeat(f64(s.d[i], n), 32, 1) * 0.5001 + 1e-12).all()
            w = q4(s.router_w[i] if i < s.L else s.head_w)
            z = f64(s.logits[i] if i < s.L else s.head_logits, n)
            xq = codes.reshape(n, -1)
            tol = (6 * s.H // 32 + 16) * 2.0 ** -23 * (np.abs(xq) @ np.abs(w).T)
            assert (np.abs(z - xq @ w.T) <= tol).all()
            if i == s.L:
                assert torch.equal(got, s.head_logits[:n])
                break
            zi = s.logits[i][:n].cpu().numpy()
            idx, wt = oracle.topk(zi, s.k)
            assert np.array_equal(idx, s.idx[i][:n].cpu().numpy())
            ref = oracle.layer(s.y[i][:n].cpu().numpy(), idx, wt, *(s.tensors[i, kd] for kd in range(3)), s.H,
                               s.wl.ffn)
            prev = f64(s.out[i], n)
            # (codes of h may round either way: a norm, as the smoke run holds it)
            assert np.linalg.norm(prev - ref) <= 1e-3 * np.linalg.norm(ref)
            loss, counts, dz = losses[i]
            assert np.array_equal(counts.cpu().numpy(), np.bincount(idx.reshape(-1), minlength=s.E))
            assert torch.isfinite(loss).all() and torch.isfinite(dz).all()
            # each row of the balance gradient sums to zero; the z loss's to 2 b lse / n
            p = np.exp(zi.astype(np.float64) - zi.max(1, keepdims=True))
            lse = zi.max(1) + np.log(p.sum(1))
            assert np.allclose(dz.cpu().numpy().sum(1), 2 * 0.001 * lse / n, rtol=1e-4, atol=1e-7)
    s.close()


def test_example_runs(capsys):
    import decoder_stack

    decoder_stack.main()
    out = capsys.readouterr().out
    assert "step 7" in out and "seed order" in out
