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
    return torch.where(m == -INF, 0.0, e / e.sum(-1, keepdim=True))


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


ALPHA = (0.1, 0.9, 1.0)


def loss_in_64_bits(d, t, lab, cf, T, alpha):
    """(loss, parts, grad_logits, its bound, grad_conf) by the formulas."""
    B, G, V = d.shape
    p, q = softmax(d, T), softmax(t, T)
    w = torch.exp(-torch.arange(G).double() / G)
    l1 = distance(d, t, T)
    label = (1 - l1 / 2).clamp(0, 1)
    x = lab.long()[..., None]
    ce = -(w * p.gather(-1, x)[..., 0].log()).sum(-1)
    c = cf.double()
    conf = -(w * (label * torch.nn.functional.logsigmoid(c) + (1 - label) * torch.nn.functional.logsigmoid(-c))).sum(-1)
    parts = torch.stack([ce, (w * l1).sum(-1), conf], dim=-1)
    s = (p - q).sign()
    hot = torch.zeros_like(p).scatter_(-1, x, 1.0)
    S = (s * p).sum(-1, keepdim=True)
    grad = (alpha[0] * (p - hot) + alpha[1] * p * (s - S)) * w[:, None] / T
    # an entry next to the kink may have either sign
    near = (p - q).abs() <= 2e-4 * p
    tol = (alpha[0] * 5e-5 * p + alpha[1] * p * (1e-4 + 1e-4 + 2 * near + 2 * (near * p).sum(-1, keepdim=True))) / T
    # and every entry by the roundings of its factors: the weight's exponential (2 + 1.2 steps of 2^-23 at
    # |x| <= 1: 7 of 2^-24), 1 / T, their product, the difference p - [v == x], two products and a sum: 13 in all
    tol = tol + 13 * 2.0 ** -24 * (alpha[0] * (p - hot).abs() + alpha[1] * p * (s - S).abs()) / T
    loss = (alpha[0] * ce if alpha[0] else 0.0) + alpha[1] * parts[:, 1] + alpha[2] * conf
    return loss, parts, grad, tol, alpha[2] * w * (torch.sigmoid(c) - label)


def check_loss(d, t, lab, cf, T=1.0, alpha=ALPHA):
    G = d.shape[1]
    loss, parts, grad, tol, gconf = loss_in_64_bits(d, t, lab, cf, T, alpha)
    ws = ds.LossWorkspace(*d.shape)
    a = [z.cuda() for z in (d, t, lab, cf)]
    got = [z.cpu().double() for z in ds.draft_loss(*a, T=T, alpha=alpha, workspace=ws)]
    assert ws.status() == 0
    fine = torch.isfinite(parts)
    assert torch.equal(got[1][~fine], parts[~fine])
    assert (got[1] - parts)[fine].abs().max() <= 3e-4 * G
    some = torch.isfinite(loss)
    assert torch.equal(got[0][~some], loss[~some])
    assert not some.any() or (got[0] - loss)[some].abs().max() <= 1e-3 * G
    over = (got[2] - grad).abs() - tol
    at = int(over.argmax())
    assert (over <= 0).all(), (at % d.shape[-1], lab.flatten()[at // d.shape[-1]], got[2].flatten()[at],
                               grad.flatten()[at], tol.flatten()[at])
    assert (got[3] - gconf).abs().max() <= 1e-4
    only = ds.draft_loss(*a, T=T, alpha=alpha, want_grads=False, workspace=ws)
    assert torch.equal(only[0].cpu().double(), got[0]) and torch.equal(only[1].cpu().double(), got[1])


def loss_inputs(B, G, V, gen):
    d = torch.randn(B, G, V, generator=gen) * 3
    return (d, d + torch.randn(B, G, V, generator=gen), torch.randint(0, V, (B, G), generator=gen, dtype=torch.int32),
            torch.randn(B, G, generator=gen))


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("share", [0.5, 0.995])
@pytest.mark.parametrize("which", ["target", "draft", "both"])
def test_draft_loss(V, share, which):
    gen = torch.Generator().manual_seed(V + 2)
    d, t, lab, cf = loss_inputs(3, 5, V, gen)
    if which != "target":
        d, lab = masked(d, share, gen)              # (labels that the mask leaves: L_ce is finite)
        lab = lab.to(torch.int32)
    if which != "draft":
        t, _ = masked(t, share, gen)
    check_loss(d, t, lab, cf, T=0.8)


@pytest.mark.parametrize("V", SIZES)
def test_draft_loss_of_empty_rows_and_masked_labels(V):
    gen = torch.Generator().manual_seed(V + 3)
    d, t, lab, cf = loss_inputs(6, 4, V, gen)
    t[0, 1] = -INF
    t[1] = -INF
    d[2, 0, int(lab[2, 0])] = -INF                  # L_ce is +inf, the gradient the formula's
    d[3, 3] = -INF
    d[4, 2] = t[4, 2] = -INF
    check_loss(d, t, lab, cf)
    check_loss(d, t, lab, cf, alpha=(0.0, 0.9, 1.0))  # then L_ce does not count


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("value", [math.nan, INF])
def test_draft_loss_of_nan_and_infinity(V, value):
    gen = torch.Generator().manual_seed(V + 4)
    d, t, lab, cf = loss_inputs(4, 3, V, gen)
    ok = [z.cpu() for z in ds.draft_loss(d.cuda(), t.cuda(), lab.cuda(), cf.cuda())]
    t[0, 1, V // 2] = value
    d[1, 2, V - 1] = value
    t[2, 0] = -INF
    t[2, 0, V // 3] = value                         # the only entry that the mask leaves
    loss, parts, g, gc = (z.cpu() for z in ds.draft_loss(d.cuda(), t.cuda(), lab.cuda(), cf.cuda()))
    assert torch.isnan(loss[:3]).all() and torch.isnan(parts[:3, 1:]).all()
    bad = torch.zeros(4, 3, dtype=torch.bool)
    bad[0, 1] = bad[1, 2] = bad[2, 0] = True
    assert torch.isnan(g[bad]).all() and torch.isnan(gc[bad]).all()
    assert torch.equal(g[~bad], ok[2][~bad]) and torch.equal(gc[~bad], ok[3][~bad])
    assert torch.equal(loss[3], ok[0][3]) and torch.equal(parts[3], ok[1][3])
