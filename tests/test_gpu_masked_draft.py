"""Draft calls with masked entries (-inf), as ``process_logits`` makes them: the labels of masked targets.

The distance is compared with 64-bit sums over the call's own logits, within 1e-4: with |x| <= 40 from the
normaliser a probability is off by three roundings of x (3 x 40 x 2^-24), the exponential's (2 + 1.2 x 40 steps of
2^-23) and its sum's (hundreds of additions of 2^-24 and the exponentials again), under 5e-5 of itself, and two rows
of probabilities sum to 2."""
import math

import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds
from semi_autoregressive_drafting_gb300 import inputs
from tests import parity
from tests.test_gpu_masked_rows import distance, masked

pytestmark = pytest.mark.gpu
INF = float("inf")
TINY, BF16, RNN = (inputs.WORKLOADS[n] for n in ("tiny_markov", "qwen3_4b_markov", "rnn_head"))
CASES = [TINY, TINY.with_(V=1001, B=3), BF16.with_(V=30000, d=256), BF16.with_(V=20003, B=2, d=64),
         BF16.with_(V=50000, B=4, d=64), BF16.with_(V=9000, B=6, d=64), BF16.with_(V=9001, B=8, d=64),
         BF16.with_(V=12000, B=70, d=64, T=0.8), BF16.with_(V=20001, B=130, d=64), RNN.with_(V=9000, B=2, d=64),
         RNN.with_(V=9001, B=9, d=64)]


def name(wl):
    return f"{wl.head}-{wl.dtype}-{wl.B}-{wl.V}"


def draft(wl, t, **kw):
    d = parity.to_dev(t)
    ws = ds.Workspace(int(wl.head == "rnn"), wl.B, wl.gamma, wl.V, wl.r, wl.d, target=d["target"] is not None)
    kw = dict(T=wl.T, seed=wl.seed, w=d["w"], target=d["target"], workspace=ws, **kw)
    if wl.head == "rnn":
        o = ds.rnn_draft(d["W1"], d["W2"], d["Wj"], d["U"], d["h"], d["x0"], **kw)
    else:
        o = ds.markov_draft(d["W1"], d["W2"], d["U"], d["x0"], h=d["h"], **kw)
    return o, ws.status()


@pytest.mark.parametrize("wl", CASES, ids=name)
@pytest.mark.parametrize("share", [0.5, 0.995])
def test_masked_targets(wl, share):
    wl = wl.with_(gamma=3, target_noise=1.0, seed=wl.V)
    t = inputs.generate(wl)
    plain, status = draft(wl, t)
    assert status == 0
    t["target"], _ = masked(t["target"], share, torch.Generator().manual_seed(wl.B))
    t["target"][0, 1] = -INF
    if wl.B > 1:
        t["target"][1, 0, wl.V // 2] = math.nan
        t["target"][1, 2] = math.nan
    a, status = draft(wl, t, want_logits=True)
    assert status == 0
    b, _ = draft(wl, t)
    want = distance(a.logits.cpu(), t["target"], wl.T)
    bad = torch.isnan(want)
    for o in (a, b):
        # the target changes nothing but the labels
        assert torch.equal(o.tokens, plain.tokens) and torch.equal(o.lse, plain.lse)
        l1, cs = o.l1.cpu().double(), o.cstar.cpu().double()
        assert torch.equal(torch.isnan(l1), bad) and torch.equal(torch.isnan(cs), bad)
        assert (l1 - want)[~bad].abs().max() <= 1e-4
        assert (cs - (1 - want / 2).clamp(0, 1))[~bad].abs().max() <= 1e-4
        assert l1[0, 1] == 2 and cs[0, 1] == 0


@pytest.mark.parametrize("wl", CASES, ids=name)
@pytest.mark.parametrize("share", [0.5, 0.995])
def test_masked_drafts(wl, share):
    # the mask of U's rows, in whole groups too, and of the target's
    wl = wl.with_(gamma=3, target_noise=1.0, seed=wl.V + 1)
    t = inputs.generate(wl)
    gen = torch.Generator().manual_seed(wl.B)
    t["U"], _ = masked(t["U"], share, gen)
    t["U"][0, 0, :wl.V // 2] = -INF
    t["U"][0, 0, wl.V - 2] = 0.0
    t["target"], _ = masked(t["target"], share, gen)
    o = parity.oracle_draft(wl, t, want_z=True)
    assert o.status == 0
    forced = torch.from_numpy(o.tokens).cuda()
    a, status = draft(wl, t, forced=forced, want_logits=True)
    assert status == 0
    parity.check_tokens_forced(a.tokens.cpu().numpy(), o)
    parity.compare_floats(a, o)
    b, status = draft(wl, t, forced=forced)
    assert status == 0
    parity.compare_floats(b, o, logits=False)
    assert torch.equal(a.tokens, b.tokens)
    assert torch.isfinite(t["U"].gather(2, a.tokens.cpu().long()[..., None]).float()).all()
    free, status = draft(wl, t)
    assert status == 0
    parity.check_tokens_free(free.tokens.cpu().numpy(), o)


@pytest.mark.parametrize("wl", CASES, ids=name)
@pytest.mark.parametrize("at", [0, 2])
def test_rows_of_u_that_nothing_is_left_of(wl, at):
    # (position 2 is the block's last)
    wl = wl.with_(gamma=3, target_noise=1.0, seed=wl.V + 2)
    t = inputs.generate(wl)
    whole, status = draft(wl, t)
    assert status == 0
    b = wl.B - 1
    t["U"][b, at] = -INF
    o, status = draft(wl, t)
    assert status == 1
    assert (o.tokens[b, at:] == -1).all()
    for name_ in ("lse", "c", "S", "l1", "cstar"):
        assert torch.isnan(getattr(o, name_)[b, at:]).all(), name_
        assert torch.equal(getattr(o, name_)[b, :at], getattr(whole, name_)[b, :at]), name_
    others = [i for i in range(wl.B) if i != b]
    for name_ in ("tokens", "lse", "c", "S", "l1", "cstar"):
        assert torch.equal(getattr(o, name_)[others], getattr(whole, name_)[others]), name_
