"""The operators together: a training step of the Markov head against 64-bit automatic
differentiation, and the example's loss."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_step_gradients_match_autograd():
    import train_markov_head as ex
    B, gamma, V, r, T, beta = 6, 4, 3000, 64, 0.9, 0.05
    g = torch.Generator().manual_seed(0)
    W1, W2 = [(torch.randn(V, r, generator=g) * 0.3).bfloat16() for _ in range(2)]
    U = torch.randn(B, gamma, V, generator=g).bfloat16()
    anchors = torch.randint(0, V, (B,), generator=g, dtype=torch.int32)
    tokens = torch.randint(0, 40, (B, gamma), generator=g, dtype=torch.int32)
    tokens[2, 2:] = -1                       # a shorter block
    loss, g1, g2, lp = ex.step(W1.cuda(), W2.cuda(), U.cuda(), anchors.cuda(), tokens.cuda(), T=T, beta=beta, top=2)

    w1, w2 = W1.double().requires_grad_(), W2.double().requires_grad_()
    cond = torch.cat([anchors[:, None], tokens[:, :-1]], dim=1).clamp(min=0).long()
    z = (U.double() + w1[cond] @ w2.t()) / T
    ln_p = z.log_softmax(-1)
    on = (tokens >= 0).double()
    logp = ln_p.gather(-1, tokens.clamp(min=0).long()[..., None])[..., 0]
    H = -(ln_p.exp() * ln_p).sum(-1)
    want = -((logp + beta * H) * on).sum() / on.sum()
    want.backward()
    assert abs(float(loss) - float(want.detach())) < 1e-4
    for got, ref in ((g1, w1.grad), (g2, w2.grad)):
        err = (got.double().cpu() - ref).norm() / ref.norm()
        # the draft's logits carry fp32 products of bf16 tables: 1e-5 of the logits, so of p
        assert float(err) < 1e-4, float(err)
    assert (lp.logp.cpu()[2, 2:] == 0).all()


def test_example_learns():
    import train_markov_head as ex
    losses = ex.main(["--steps", "12", "--vocab", "5000", "--batch", "32"])
    assert losses[-1] < losses[0] - 0.5, losses
