"""One workspace of the token log probabilities serves calls of other sizes, in any order.

Small calls count each row's finished blocks in the workspace.  What a call of fewer rows leaves there
must not be in the place of those counters: rows would be merged too early or never.  The outputs hold
NaN before every call, and every call is compared with one on a workspace of its own."""
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds


def outputs(N, top):
    nan = float("nan")
    o = ds.LogprobOutput(torch.full((N,), nan), torch.full((N, 2), nan), torch.full((N,), nan),
                         torch.full((N,), -9, dtype=torch.int32),
                         torch.full((N, top), -9, dtype=torch.int32) if top else None,
                         torch.full((N, top), nan) if top else None)
    return ds.LogprobOutput(**{k: v if v is None else v.cuda() for k, v in vars(o).items()})


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("top", [0, 6])
@pytest.mark.parametrize("calls", [
    [(77, 50021), (8, 50021), (77, 50021)],
    [(131, 32000), (16, 32000), (131, 32000), (1, 32000), (70, 32000)],
    [(512, 8000), (8, 8000), (512, 8000)],
    # the most rows that are counted, before and after calls in two launches and of one-chunk rows
    [(1024, 4094), (3, 4094), (1024, 4094), (1000, 60000), (1024, 4094), (2000, 900), (1024, 4094)],
])
def test_one_workspace_for_calls_of_other_sizes(calls, top, dtype):
    ws = ds.LogprobWorkspace(max(n for n, _ in calls), max(v for _, v in calls), top)
    for i, (N, V) in enumerate(calls):
        g = torch.Generator(device="cuda").manual_seed(i + N + V)
        # rows one element past a 16-byte boundary, a padded stride
        z = torch.randn(N * (V + 3) + 1, generator=g, device="cuda").mul_(3).to(dtype)[1:].view(N, V + 3)[:, :V]
        t = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
        got = ds.token_logprobs(z, t, top=top, workspace=ws, out=outputs(N, top))
        own = ds.token_logprobs(z, t, top=top, out=outputs(N, top))
        for name, want in vars(own).items():
            if want is not None:
                assert not torch.isnan(want).any() and torch.equal(getattr(got, name), want), (i, N, V, name)
        assert ws.status() == 0
