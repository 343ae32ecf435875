"""Verification where a mask leaves nothing of a row, of the target (a correction's or the bonus's) or of the draft."""
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds
from semi_autoregressive_drafting_gb300 import inputs

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("V", [4096, 4001, 20003, 40000])
def test_rows_that_nothing_is_left_of(V, oracle_mod):
    B, G = 8, 4
    t = inputs.verify_inputs(B, G, V, seed=V, target_noise=0.0, tokens="argmax")   # (accepted: p and q agree)
    zd, zt, tok = t["draft_logits"], t["target_logits"], t["draft_tokens"]
    zt[0, 0] = -INF                                     # the first position's row: no correction to draw
    zt[1, 2] = -INF                                     # a later one
    zt[2, G] = -INF                                     # the bonus
    zt[3] = -INF
    zd[4, 1] = -INF                                     # of the draft: rejected, the correction from q
    zd[5, 1] = zt[5, 1] = -INF
    zd[6, 3, int(tok[6, 3])] = -INF                     # a drafted token that the draft masks: q / p is infinite
    zt[7, 1, int(tok[7, 1])] = -INF                     # one that the target masks: rejected
    ws = ds.VerifyWorkspace(B, G, V)
    n, out = ds.verify(zd.cuda(), zt.cuda(), tok.cuda(), seed=3, workspace=ws)
    assert ws.status() == 0
    n, out = n.cpu(), out.cpu()
    assert n.tolist() == [0, 2, G, 0, 1, 1, G, 1]
    for b, k in ((0, 0), (1, 2), (2, G), (3, 0), (5, 1)):
        assert (out[b, :k] == tok[b, :k]).all() and (out[b, k:] == -1).all()
    assert out[4, 1] >= 0 and out[6, G] >= 0 and out[7, 1] >= 0 and out[7, 1] != tok[7, 1]
    ref = oracle_mod.verify(gamma=G, T=1.0, seed=3, draft_logits=zd.numpy(), target_logits=zt.numpy(),
                            draft_tokens=tok.numpy())
    assert (n.numpy() == ref.n_accepted).all() and (out.numpy() == ref.tokens).all()
    # the workspace is ready for the next call
    again = ds.verify(zd.cuda(), zt.cuda(), tok.cuda(), seed=3, workspace=ws)
    assert torch.equal(again[0].cpu(), n) and torch.equal(again[1].cpu(), out)


@pytest.mark.parametrize("V", [4096, 4001, 40000])
def test_rows_with_nan(V):
    # NaN is met wherever it stands, also where a mask leaves nothing else of a thread's entries
    B, G = 5, 3
    t = inputs.verify_inputs(B, G, V, seed=V + 1, target_noise=0.0, tokens="argmax")
    zd, zt, tok = t["draft_logits"], t["target_logits"], t["draft_tokens"]
    nan = float("nan")
    zt[0, 1, V // 2] = nan
    keep = zt[1, 2, int(tok[1, 2])].clone()
    zt[1, 2] = -INF
    zt[1, 2, int(tok[1, 2])], zt[1, 2, (int(tok[1, 2]) + 1501) % V] = keep, nan
    zt[2, G] = -INF
    zt[2, G, 7] = nan
    zd[3, 0, V - 1] = nan
    zt[4] = nan
    n, out = (x.cpu() for x in ds.verify(zd.cuda(), zt.cuda(), tok.cuda(), seed=3))
    assert n.tolist() == [1, 2, G, 0, 0]
    for b in (0, 1, 2, 4):
        assert (out[b, int(n[b]):] == -1).all() and (out[b, :int(n[b])] == tok[b, :int(n[b])]).all()
    assert out[3, 0] >= 0 and (out[3, 1:] == -1).all()
