"""Trains the Markov head's two tables (Eq 5) by the likelihood of given tokens.

The parallel backbone's base logits U are fixed; the head adds B_k = W1[x_{k-1}] W2.  One step runs,
all on the library's kernels:

  forward   e = W1[x_{k-1}]                        ds.embedding
            z = U + e W2                           ds.markov_draft, teacher-forced (also e's lookup)
            log p(x_k), entropy, alternatives      ds.token_logprobs
  backward  dL/dz                                  ds.token_logprobs_grad
            dL/de, dL/dW2                          ds.bias_grad
            dL/dW1                                 ds.embedding_grad

for L = mean over the given tokens of -log p(x_k) - beta H_k, and updates fp32 master copies of the
tables by gradient descent.  The data is synthetic: tokens follow a fixed random successor table, so
that the head has something to learn.

  python examples/train_markov_head.py [--steps 20] [--vocab 32000] [--batch 32]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import semi_autoregressive_drafting_gb300 as ds


def batch(gen, succ, B, gamma):
    """Anchors [B] and tokens [B, gamma]: each token's successor nine times in ten, else any."""
    V = succ.numel()
    x = torch.randint(0, V, (B,), generator=gen, device="cuda")
    anchors, tokens = x, []
    for _ in range(gamma):
        other = torch.randint(0, V, (B,), generator=gen, device="cuda")
        x = torch.where(torch.rand(B, generator=gen, device="cuda") < 0.9, succ[x], other)
        tokens.append(x)
    return anchors.to(torch.int32), torch.stack(tokens, dim=1).to(torch.int32)


def step(W1, W2, U, anchors, tokens, *, T=1.0, beta=0.0, seed=0, top=0):
    """One forward and backward pass with bf16 tables W1, W2 [V, r] and base logits U [B, gamma, V].

    Returns (L, dL/dW1, dL/dW2, the LogprobOutput).  Tokens of -1 (ragged blocks) have no part in L."""
    B, gamma, V = U.shape
    cond = torch.cat([anchors[:, None], tokens[:, :-1]], dim=1).clamp(min=0).contiguous()
    given = tokens.clamp(min=0)
    z = ds.markov_draft(W1, W2, U, anchors, T=T, seed=seed, forced=given, want_logits=True).logits
    e = ds.embedding(W1, cond)
    lp = ds.token_logprobs(z, tokens, T=T, top=top)
    on = (tokens >= 0).float()
    n = on.sum().clamp(min=1.0)
    loss = -((lp.logp + beta * lp.entropy) * on).sum() / n
    g = ds.token_logprobs_grad(z, tokens, lp.norm, T=T, grad_logp=-on / n, grad_entropy=-beta * on / n,
                               entropy=lp.entropy, out=z)
    grad_e, grad_W2 = ds.bias_grad(g, e, W2)
    grad_W1 = ds.embedding_grad(grad_e, cond, V)
    return loss, grad_W1, grad_W2, lp


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--batch", type=int, default=32)
    ap.add_argument("--gamma", type=int, default=7)
    ap.add_argument("--rank", type=int, default=64)
    ap.add_argument("--lr", type=float, default=None, help="step size (default: 20 per token of the batch)")
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    V, r, B = a.vocab, a.rank, a.batch
    # few successors' chains, so that a short run meets its tokens again
    succ = torch.randint(0, min(V, 64), (V,), generator=gen, device="cuda")
    W1, W2 = [torch.randn(V, r, generator=gen, device="cuda") * 0.3 for _ in range(2)]
    U = torch.randn(B, a.gamma, V, generator=gen, device="cuda").bfloat16()
    lr = a.lr if a.lr is not None else 20.0 * B * a.gamma / 224
    losses = []
    for i in range(a.steps):
        anchors, tokens = batch(gen, succ, B, a.gamma)
        loss, g1, g2, lp = step(W1.bfloat16(), W2.bfloat16(), U, anchors, tokens, seed=i, top=3)
        W1.add_(g1, alpha=-lr)
        W2.add_(g2, alpha=-lr)
        losses.append(float(loss))
        print(f"step {i:3d}  loss {losses[-1]:.4f}  entropy {float(lp.entropy.mean()):.3f}  "
              f"given token first {float((lp.rank == 1).float().mean()):.2f}")
    return losses


if __name__ == "__main__":
    main()
