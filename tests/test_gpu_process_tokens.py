"""The ends of the tokens' type, wherever a request holds one, make that request's rows NaN and no other's."""
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("token", [2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1, 2 ** 24])
@pytest.mark.parametrize("H", [4, 70000])
def test_ends_of_the_type(token, H):
    B, R, V = 5, 3, 20011
    g = torch.Generator().manual_seed(H)
    z = torch.randn(B, R, V, generator=g).cuda()
    x = dict(history=torch.randint(0, V, (B, H), generator=g, dtype=torch.int32).cuda(),
             drafted=torch.randint(0, V, (B, R - 1), generator=g, dtype=torch.int32).cuda(),
             bias_tokens=torch.randint(0, V, (B, 3), generator=g, dtype=torch.int32).cuda(),
             bias=torch.randn(B, 3, generator=g).cuda(), repetition=torch.full((B,), 1.5, device="cuda"))
    whole = ds.process_logits(z, **x)
    x["history"][0, H - 1] = token
    x["drafted"][1, 0] = token
    x["bias_tokens"][2, 1] = token
    got = ds.process_logits(z, **x)
    assert torch.isnan(got[:3]).all() and torch.equal(got[3:], whole[3:])
    w = {k: x[k] for k in ("history", "drafted", "repetition")}
    grad = ds.process_logits_grad(torch.ones_like(z), z, **w)
    assert torch.isnan(grad[:2]).all() and torch.isfinite(grad[2:]).all()
