"""The operators around the logits together: a grammar and penalties on target and draft, the target's
alternatives, distillation from them, the gradient back through the processors and on to W1 and W2."""
import math

import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds
from tests.test_gpu_process import allowed_rows, dev, make

pytestmark = pytest.mark.gpu


def test_distilling_the_head_under_a_grammar_matches_autograd():
    B, G, V, r, K, T = 5, 4, 3000, 64, 24, 0.8
    alpha = (0.4, 0.6)
    tz, x = make(B, G, V, 60, seed=3, dtype=torch.bfloat16, nb=5, masked=3)
    g = torch.Generator().manual_seed(4)
    x["mask"][:, :8] = -1                                            # (every row keeps some entries)
    x = {k: v for k, v in x.items() if k not in ("presence", "frequency")}
    W1, W2 = [(torch.randn(V, r, generator=g) * 0.3).bfloat16() for _ in range(2)]
    U = torch.randn(B, G, V, generator=g).bfloat16()
    anchors = torch.randint(0, V, (B,), generator=g, dtype=torch.int32)
    given = x["drafted"] = torch.randint(0, V, (B, G - 1), generator=g, dtype=torch.int32)
    tokens = torch.cat([given, torch.zeros(B, 1, dtype=torch.int32)], dim=1)
    cond = torch.cat([anchors[:, None], given], dim=1)
    weight = (torch.rand(B, G, generator=g) / (B * G))
    weight[1, 2:] = 0.0

    # the teacher: the target's processed logits and their K most likely entries
    tools = dev(x)
    tq = ds.process_logits(tz.cuda(), dtype=torch.float32, **tools)
    top = ds.token_logprobs(tq, tokens.cuda(), T=T, top=K)
    # the student: the draft's logits under the same tools
    z = ds.markov_draft(W1.cuda(), W2.cuda(), U.cuda(), anchors.cuda(), forced=tokens.cuda(), want_logits=True).logits
    grad_tools = {k: v for k, v in tools.items() if k not in ("bias_tokens", "bias")}
    y = ds.process_logits(z, **tools)
    o = ds.distill_loss(y, top.top_ids, top.top_logp, T=T, alpha=alpha, weight=weight.cuda())
    gz = ds.process_logits_grad(o.grad_logits, z, out=o.grad_logits, **grad_tools)
    e = ds.embedding(W1.cuda(), cond.cuda())
    ge, g2 = ds.bias_grad(gz, e, W2.cuda())
    g1 = ds.embedding_grad(ge, cond.cuda(), V)

    # the same in 64 bits by automatic differentiation
    w1, w2 = W1.double().requires_grad_(), W2.double().requires_grad_()
    rz = U.double() + w1[cond.long()] @ w2.t()
    seen = torch.zeros(B, G, V, dtype=torch.bool)
    bias = torch.zeros(B, 1, V, dtype=torch.float64)
    for b in range(B):
        for t in x["history"][b, :int(x["lengths"][b])].tolist():
            seen[b, :, t] = True
        for k in range(1, G):
            seen[b, k:, int(given[b, k - 1])] = True
        for t, v in zip(x["bias_tokens"][b].tolist(), x["bias"][b].tolist()):
            if t >= 0:
                bias[b, 0, t] += v
    ok = allowed_rows(x, B * G, V).view(B, G, V)
    rho = x["repetition"].double()[:, None, None]

    def tool(v):
        v = torch.where(seen, torch.where(v > 0, v / rho, v * rho), v) + bias
        return v.masked_fill(~ok, -math.inf)
    tlp = torch.log_softmax(tool(tz.double()) / T, -1)
    lq, ids = top.top_logp.double().cpu(), top.top_ids.long().cpu()
    have = ids >= 0
    assert torch.allclose(lq[have], tlp.gather(-1, ids.clamp(min=0))[have], atol=1e-5)
    lp = torch.log_softmax(tool(rz) / T, -1)
    hot = torch.zeros(B, G, V, dtype=torch.bool)
    hot.view(-1, V)[torch.arange(B * G)[:, None].expand(-1, K)[have.view(-1, K)], ids.view(-1, K)[have.view(-1, K)]] = True
    pr = (lp.exp() * ~hot).sum(-1)
    pj = torch.where(have, lp.gather(-1, ids.clamp(min=0)), torch.zeros_like(lq))
    q = torch.where(have, lq.exp(), torch.zeros_like(lq))
    qr = 1 - q.sum(-1)
    kl = (q * torch.where(have, lq - pj, torch.zeros_like(lq))).sum(-1) + qr * (qr.log() - pr.log())
    l1 = (torch.where(have, pj.exp(), torch.zeros_like(lq)) - q).abs().sum(-1) + (pr - qr).abs()
    loss = (weight.double() * (alpha[0] * kl + alpha[1] * l1)).sum()
    loss.backward()
    assert abs(float(o.loss.sum()) - float(loss.detach())) < 1e-5
    for got, ref in ((g1, w1.grad), (g2, w2.grad)):
        err = (got.double().cpu() - ref).norm() / ref.norm()
        # the draft's logits carry fp32 products of bf16 tables: 1e-5 of the logits, so of p
        assert float(err) < 1e-4, float(err)
    # nothing flows into masked entries
    assert (gz.cpu()[~ok] == 0).all()
