"""Logits and output as ranges of columns of one buffer give what separate ones give, and touch nothing else."""
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,left,mid,right", [(8192, 0, 0, 0), (9001, 3, 5, 2), (20011, 8, 0, 5)])
@pytest.mark.parametrize("swap", [False, True])
def test_columns_of_one_buffer(V, left, mid, right, swap, dtype):
    B, R = 3, 2
    g = torch.Generator().manual_seed(V)
    W = left + 2 * V + mid + right
    buf = torch.full((B, R, W), 7.0, dtype=dtype, device="cuda")
    a, b = buf[..., left:left + V], buf[..., left + V + mid:left + 2 * V + mid]
    z, out = (b, a) if swap else (a, b)
    # (the same logits at the same places within 16 bytes, in a buffer of their own)
    data = torch.zeros_like(buf)[..., left + V + mid:left + 2 * V + mid] if swap else torch.zeros_like(buf)[..., left:left + V]
    data.copy_((torch.randn(B, R, V, generator=g) * 3).to(dtype))
    z.copy_(data)
    edges = torch.cat([buf[..., :left], buf[..., left + V:left + V + mid], buf[..., W - right:]], dim=-1).clone()

    def untouched():
        now = torch.cat([buf[..., :left], buf[..., left + V:left + V + mid], buf[..., W - right:]], dim=-1)
        return torch.equal(now, edges) and torch.equal(z, data)
    x = dict(history=torch.randint(0, V, (B, 500), generator=g, dtype=torch.int32).cuda(),
             repetition=torch.full((B,), 1.25, device="cuda"),
             mask=torch.randint(-2 ** 31, 2 ** 31 - 1, (B * R, (V + 31) // 32), generator=g).to(torch.int32).cuda())
    want = ds.process_logits(data, **x)
    assert torch.equal(ds.process_logits(z, out=out, **x), want) and untouched()
    want = ds.process_logits_grad(data, data, **x)
    assert torch.equal(ds.process_logits_grad(z, data, out=out, **x), want) and untouched()
    K = 20
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(B * R)]).view(B, R, K).to(torch.int32).cuda()
    lq = torch.log_softmax(torch.randn(B, R, K + 1, generator=g), dim=-1)[..., :K].contiguous().cuda()
    want = ds.distill_loss(data, ids, lq, T=0.8, alpha=(0.5, 0.5))
    o = ds.DistillOutput(torch.empty_like(want.loss), torch.empty_like(want.parts), torch.empty_like(want.norm), out)
    got = ds.distill_loss(z, ids, lq, T=0.8, alpha=(0.5, 0.5), out=o)
    assert torch.equal(got.loss, want.loss) and torch.equal(got.grad_logits, want.grad_logits) and untouched()
    w = torch.ones(B, R, device="cuda")
    want = ds.distill_grad(data, ids, lq, want.norm, w, T=0.8, alpha=(0.5, 0.5))
    assert torch.equal(ds.distill_grad(z, ids, lq, got.norm, w, T=0.8, alpha=(0.5, 0.5), out=out), want) and untouched()
