"""A row's results do not depend on the rows beside it: small calls (one launch, short segments) and
large ones (two launches) give the same bits."""
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("N,V,few,off", [(600, 30000, 60, 0), (600, 30000, 1, 0), (80, 151936, 20, 0),
                                         (3000, 5001, 300, 1), (40, 262144, 3, 0), (9000, 1000, 1000, 0),
                                         (700, 20003, 7, 3)])
def test_rows_alone_and_in_a_large_call(N, V, few, off, top, dtype):
    g = torch.Generator(device="cuda").manual_seed(N + V + few)
    # one row stride throughout, so that every row starts at the same place of its 16 bytes
    ld = (V + off + 7) // 8 * 8
    z = torch.randn(N, ld, generator=g, device="cuda").mul_(3).to(dtype)[:, off:off + V]
    z[::7, ::3] = -float("inf")
    z[::11, 5:90] = torch.finfo(dtype).min
    t = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    assert N * V * z.element_size() > 16 << 20 >= few * V * z.element_size()
    many = ds.token_logprobs(z, t, T=0.7, top=top)
    for i in range(0, min(N, 40 * few), few):
        some = ds.token_logprobs(z[i:i + few], t[i:i + few], T=0.7, top=top)
        for name, want in vars(many).items():
            if want is not None:
                got = getattr(some, name)
                assert torch.equal(got, want[i:i + few]), (i, name, int((got != want[i:i + few]).sum()))
