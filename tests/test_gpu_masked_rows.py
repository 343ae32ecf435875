"""Rows whose entries a mask rules out (-inf), as ``process_logits`` makes them, in the calls that take whole rows.

Tolerances.  With |x| <= 40 the logits' distance from the normaliser, a probability is off by three roundings of
x (3 x 40 x 2^-24), the exponential's own error (2 + 1.2 x 40 steps of 2^-23) and its normaliser's sum (V / 256
additions per thread at most, and the exponentials' errors again): under 5e-5 of itself.  A distance of two rows sums
probabilities of 1 each: 1e-4; a draft loss has gamma of them, weighted by 1 at most."""
import math

import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

pytestmark = pytest.mark.gpu
INF = float("inf")


def masked(z, share, gen):
    """z with a share of its entries at -inf, but for one of each row."""
    off = torch.rand(z.shape, generator=gen) < share
    keep = torch.randint(0, z.shape[-1], z.shape[:-1], generator=gen)
    off.scatter_(-1, keep[..., None], False)
    return z.masked_fill(off, -INF), keep


def softmax(z, T=1.0):
    """In 64 bits; a row that is -inf everywhere has no probabilities."""
    z = z.double() / T
    m = z.amax(-1, keepdim=True)
    e = (z - torch.where(m == -INF, 0.0, m)).exp()
    s = e.sum(-1, keepdim=True)
    return torch.where(s > 0, e / s, 0.0)


def distance(d, t, T=1.0):
    p, q = softmax(d, T), softmax(t, T)
    l1 = (p - q).abs().sum(-1)
    return torch.where((p.sum(-1) == 0) | (q.sum(-1) == 0), 2.0, l1)


SIZES = [7, 4096, 4001, 20003, 70000]


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("share", [0.5, 0.995])
@pytest.mark.parametrize("which", ["target", "draft", "both"])
def test_tv_label(V, share, which):
    N, T = 9, 0.8
    gen = torch.Generator().manual_seed(V)
    d = torch.randn(N, V, generator=gen) * 3
    t = d + torch.randn(N, V, generator=gen)
    if which != "target":
        d, _ = masked(d, share, gen)
    if which != "draft":
        t, _ = masked(t, share, gen)
    cs, l1 = ds.tv_label(d.cuda(), t.cuda(), T=T)
    want = distance(d, t, T)
    assert (l1.cpu().double() - want).abs().max() <= 1e-4
    assert (cs.cpu().double() - (1 - want / 2).clamp(0, 1)).abs().max() <= 1e-4


@pytest.mark.parametrize("V", SIZES)
def test_tv_label_of_empty_rows_and_nan(V):
    gen = torch.Generator().manual_seed(V + 1)
    d, t = torch.randn(6, V, generator=gen), torch.randn(6, V, generator=gen)
    t[0] = -INF
    d[1] = -INF
    d[2] = t[2] = -INF
    t[3, V // 2] = math.nan
    d[4, V - 1] = INF
    cs, l1 = (x.cpu() for x in ds.tv_label(d.cuda(), t.cuda()))
    assert (l1[:3] == 2).all() and (cs[:3] == 0).all()
    assert torch.isnan(l1[3:5]).all() and torch.isnan(cs[3:5]).all()
    assert abs(float(l1[5]) - float(distance(d[5], t[5]))) <= 1e-4
