"""Token log probabilities of a single row without leading dimensions."""
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds


@pytest.mark.gpu
@pytest.mark.parametrize("top", [0, 3])
def test_one_row_without_leading_dimensions(top):
    g = torch.Generator().manual_seed(1)
    z = torch.randn(1, 3000, generator=g).cuda()
    t = torch.tensor([17], dtype=torch.int32).cuda()
    want = ds.token_logprobs(z, t, top=top)
    got = ds.token_logprobs(z[0], t[0], top=top)
    assert got.logp.shape == () and got.norm.shape == (2,)
    for name, w in vars(want).items():
        assert w is None or torch.equal(getattr(got, name), w[0]), name
    one = torch.ones(1, device="cuda")
    grad = ds.token_logprobs_grad(z, t, want.norm, grad_logp=one)
    assert torch.equal(ds.token_logprobs_grad(z[0], t[0], got.norm, grad_logp=one[0]), grad[0])


@pytest.mark.gpu
def test_an_output_without_alternatives_is_refused_where_they_are_asked_for():
    z = torch.randn(2, 100, device="cuda")
    t = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        ds.token_logprobs(z, t, top=2, out=ds.token_logprobs(z, t))
