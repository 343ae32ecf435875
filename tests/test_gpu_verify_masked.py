"""Verification of targets whose entries a grammar has masked (-inf), against the oracle."""
import numpy as np
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [4096, 4001, 20003])
@pytest.mark.parametrize("share", [0.5, 0.99])
def test_masked_targets(V, share, oracle_mod):
    B, G = 8, 5
    g = torch.Generator().manual_seed(V)
    zd = torch.randn(B, G, V, generator=g)
    zt = torch.cat([zd + 0.3 * torch.randn(B, G, V, generator=g), torch.randn(B, 1, V, generator=g)], dim=1)
    off = torch.rand(B, G + 1, V, generator=g) < share
    off[0] = True
    off[0, :, 17] = False                                            # one entry left
    zt[off] = -np.inf
    # drafted tokens that the target allows, but for one request's second
    tok = torch.stack([torch.stack([torch.nonzero(~off[b, j])[(b + j) % 7 if b else 0, 0] for j in range(G)])
                       for b in range(B)]).to(torch.int32)
    tok[3, 1] = int(torch.nonzero(off[3, 1])[0, 0])
    n, out = ds.verify(zd.cuda(), zt.cuda(), tok.cuda(), seed=9)
    ref = oracle_mod.verify(gamma=G, T=1.0, seed=9, draft_logits=zd.numpy(), target_logits=zt.numpy(),
                            draft_tokens=tok.numpy())
    assert (n.cpu().numpy() == ref.n_accepted).all()
    assert (out.cpu().numpy() == ref.tokens).all()
    assert int(n[3]) <= 1
