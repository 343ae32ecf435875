"""Masks of the type's lowest number, whose scaled value is -inf in units of log2, give what masks of -inf give."""
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds
from semi_autoregressive_drafting_gb300 import inputs
from tests.test_gpu_masked_draft import CASES, draft, name
from tests.test_gpu_masked_rows import loss_inputs, masked

pytestmark = pytest.mark.gpu
INF = float("inf")


def lowest(z):
    return torch.where(z == -INF, torch.finfo(z.dtype).min, z)


@pytest.mark.parametrize("V", [7, 4096, 4001, 40000])
@pytest.mark.parametrize("T", [1.0, 0.8, 2.0])
def test_labels_and_losses(V, T):
    gen = torch.Generator().manual_seed(V)
    d, t, lab, cf = loss_inputs(3, 4, V, gen)
    d, lab = masked(d, 0.995, gen)
    t, _ = masked(t, 0.995, gen)
    lab = lab.to(torch.int32).cuda()
    out = []
    for x, y in ((d, t), (lowest(d), lowest(t))):
        x, y = x.cuda(), y.cuda()
        out.append([*ds.tv_label(x.view(-1, V), y.view(-1, V), T=T), *ds.draft_loss(x, y, lab, cf.cuda(), T=T)])
    for a, b in zip(*out):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("V", [4096, 4001, 40000])
@pytest.mark.parametrize("T", [1.0, 0.8, 2.0])
def test_verify(V, T):
    B, G = 16, 5
    gen = torch.Generator().manual_seed(V + 1)
    d = torch.randn(B, G, V, generator=gen)
    t = torch.cat([d + 0.3 * torch.randn(B, G, V, generator=gen), torch.randn(B, 1, V, generator=gen)], dim=1)
    t, keep = masked(t, 0.995, gen)
    d, _ = masked(d, 0.5, gen)
    d.scatter_(2, keep[:, :G, None], 0.0)
    tok = keep[:, :G].to(torch.int32).cuda()
    a, b = (ds.verify(x.cuda(), y.cuda(), tok, T=T, seed=4) for x, y in ((d, t), (lowest(d), lowest(t))))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    n, out = a[0].cpu(), a[1].cpu()
    assert (n > 0).any()
    for i in range(B):
        assert t[i, int(n[i]), int(out[i, int(n[i])])] > -INF


@pytest.mark.parametrize("wl", CASES, ids=name)
def test_drafts(wl):
    wl = wl.with_(gamma=3, target_noise=1.0, seed=wl.V + 3)
    t = inputs.generate(wl)
    gen = torch.Generator().manual_seed(wl.B)
    t["U"], _ = masked(t["U"], 0.99, gen)
    t["U"][0, 0, :wl.V // 2] = -INF
    t["U"][0, 0, wl.V - 2] = 0.0
    t["target"], _ = masked(t["target"], 0.99, gen)
    a, status = draft(wl, t)
    assert status == 0
    b, status = draft(wl, {**t, "U": lowest(t["U"]), "target": lowest(t["target"])})
    assert status == 0
    for k in ("tokens", "lse", "l1", "cstar"):
        assert torch.equal(getattr(a, k), getattr(b, k)), k
    assert torch.isfinite(a.lse).all()
