"""Teacher's probabilities that fp32 does not hold: they count as 0, but for a token that the student masks."""
import math

import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.mark.parametrize("copies", [1, 525])   # on the chip, and the loss alone in two launches
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rest", [True, False])
def test_small_probabilities(copies, dtype, rest):
    V, K = 8000 if dtype == torch.float32 else 16000, 4
    g = torch.Generator().manual_seed(4)
    z = torch.randn(4, V, generator=g)
    ids = torch.tensor([[5, 77, 4001, V - 1]] * 4, dtype=torch.int32)
    lq = torch.tensor([[math.log(0.75), -90.0, -500.0, -3.0]] * 4)
    z[0, 77] = -INF
    z[1, 4001] = -INF
    z[2, 100:200] = -INF
    ids[3, 1], lq[3, 1] = -1, -INF
    z[3, 77] = -INF
    z = z.to(dtype)
    many = [x.repeat(copies, 1).cuda() for x in (z, ids, lq)]
    p = torch.log_softmax(z.double(), dim=-1)
    q = lq.double().exp()
    lp = torch.where(ids >= 0, p.gather(1, ids.long().clamp(min=0)), 0.0)
    kl = torch.where(q > 1e-30, q * (lq.double() - lp), 0.0).sum(1)
    if rest:
        qr = 1 - q.sum(1)
        hidden = torch.zeros(4, V + 1, dtype=torch.bool).scatter_(1, torch.where(ids >= 0, ids, V).long(), True)
        kl = kl + qr * (qr.log() - torch.logsumexp(p.masked_fill(hidden[:, :V], -INF), dim=-1))
    for grad in (False, True):
        o = ds.distill_loss(*many, rest=rest, want_grad=grad)
        got = o.parts.cpu().double()[:, 0].view(copies, 4)
        assert (got == got[0]).all()
        assert got[0, 0] == INF and got[0, 1] == INF
        # ln p and the outcomes to some 2^-20 (see the distillation's own tests)
        assert (got[0, 2:] - kl[2:]).abs().max() <= 2.0 ** -18 * (1 + math.log(V))
        if grad:
            assert torch.isfinite(o.grad_logits.float()).all()
