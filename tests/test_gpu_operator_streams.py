"""The plans on other streams than the memory's own: what a pending call uses is not handed out again,
and a workspace is clear before its first use."""
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

pytestmark = pytest.mark.gpu
PAUSE = 400_000_000    # cycles: some 200 ms


def test_memory_of_a_pending_call_is_not_reused():
    N, V, D = 300, 2000, 64
    g = torch.randn(N, D, device="cuda")
    t = torch.randint(0, V, (N,), dtype=torch.int32, device="cuda")
    out = torch.empty(V, D, device="cuda")
    ws = ds.EmbeddingGradWorkspace(N, V, D)
    s = torch.cuda.Stream()
    ds.embedding_grad(g, t, V)                      # (the kernels are loaded)
    with torch.cuda.stream(s):
        torch.cuda._sleep(1)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(PAUSE)
    ds.embedding_grad(g, t, V, out=out, workspace=ws, stream=s)
    taken = {x.data_ptr() for x in (g, t, out, ws.buf)}
    sizes = [(x.shape, x.dtype) for x in (g, t, out, ws.buf)]
    assert not s.query()                            # the call is still to come
    del g, t, out, ws
    new = [torch.empty(shape, dtype=dt, device="cuda") for shape, dt in sizes]
    assert not taken & {x.data_ptr() for x in new}
    s.synchronize()


def test_first_run_on_another_stream_finds_a_clear_workspace():
    N, V = 40, 20000
    z = torch.randn(N, V, device="cuda")
    t = torch.randint(0, V, (N,), dtype=torch.int32, device="cuda")
    want = ds.token_logprobs(z, t, top=3)
    s = torch.cuda.Stream()
    dirty = torch.full((ds.LogprobWorkspace(N, V, 3).nbytes,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del dirty                                       # the plan's workspace takes its place
    torch.cuda._sleep(PAUSE)
    plan = ds.LogprobPlan(z, t, top=3)              # cleared behind the pause
    got = plan.run(s)
    s.synchronize()
    for name, w in vars(want).items():
        assert torch.equal(getattr(got, name), w), name
    assert plan.workspace.status() == 0


@pytest.mark.parametrize("kind", ["logprob", "embed_grad"])
def test_run_on_several_streams_in_turn(kind):
    N, V, D = 500, 3000, 40
    t = torch.randint(0, V, (N,), dtype=torch.int32, device="cuda")
    if kind == "logprob":
        plan = ds.LogprobPlan(torch.randn(N, V, device="cuda"), t, top=2)
        first = lambda: plan.out.logp
    else:
        plan = ds.EmbeddingGradPlan(torch.randn(N, D, device="cuda"), t, V)
        first = lambda: plan.out
    plan.run()
    want = first().clone()
    for _ in range(2):
        for s in (torch.cuda.Stream(), torch.cuda.Stream()):
            torch.cuda.synchronize()
            first().fill_(7.0)
            torch.cuda.synchronize()
            plan.run(s)
            s.synchronize()
            assert torch.equal(first(), want)
