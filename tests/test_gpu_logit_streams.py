"""Processors and distillation on other streams than the memory's own, and in calls that are split differently."""
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

pytestmark = pytest.mark.gpu
PAUSE = 400_000_000    # cycles: some 200 ms


def request(B, R, V, H, nb, seed):
    g = torch.Generator().manual_seed(seed)
    ints = lambda *s: torch.randint(-1, V, s, generator=g).to(torch.int32).cuda()
    real = lambda *s: (0.5 + torch.rand(s, generator=g)).cuda()
    return dict(history=ints(B, H), drafted=ints(B, R - 1), repetition=real(B), presence=real(B), frequency=real(B),
                bias_tokens=ints(B, nb), bias=real(B, nb),
                mask=torch.randint(-2 ** 31, 2 ** 31, (3, (V + 31) // 32), generator=g).to(torch.int32).cuda(),
                mask_rows=torch.randint(-1, 3, (B, R), generator=g).to(torch.int32).cuda())


def teacher(N, V, K, seed):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, V, generator=g) * 3
    logq, ids = torch.log_softmax(torch.randn(N, V, generator=g) * 3, -1).topk(K, -1)
    return z.cuda(), ids.to(torch.int32).cuda(), logq.cuda()


def test_memory_of_a_pending_call_is_not_reused():
    z, ids, logq = teacher(64, 3000, 8, 1)
    r = request(64, 1, 3000, 50, 4, 2)
    r["mask_rows"] = r["mask_rows"].view(64)
    s = torch.cuda.Stream()
    ds.distill_loss(z, ids, logq)
    ds.process_logits(z, **r)
    with torch.cuda.stream(s):
        torch.cuda._sleep(1)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(PAUSE)
    y = torch.empty_like(z)
    ds.process_logits(z, out=y, stream=s, **r)
    o = ds.distill_loss(y, ids, logq, stream=s)
    used = [z, ids, logq, y, *r.values()]
    taken = {x.data_ptr() for x in used if x.numel()}
    sizes = [(x.shape, x.dtype) for x in used if x.numel()]
    assert not s.query()                            # the calls are still to come
    del z, ids, logq, y, r, used
    new = [torch.empty(shape, dtype=dt, device="cuda") for shape, dt in sizes]
    assert not taken & {x.data_ptr() for x in new}
    s.synchronize()
    assert o.loss.shape == (64,)


def test_first_run_on_another_stream_finds_a_clear_workspace():
    z, ids, logq = teacher(40, 20000, 16, 3)
    want = ds.distill_loss(z, ids, logq)
    s = torch.cuda.Stream()
    dirty = torch.full((ds.DistillWorkspace(40, 20000, 16).nbytes,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del dirty                                       # the plan's workspace takes its place
    torch.cuda._sleep(PAUSE)
    plan = ds.DistillPlan(z, ids, logq)             # cleared behind the pause
    got = plan.run(s)
    s.synchronize()
    for name, w in vars(want).items():
        assert torch.equal(getattr(got, name), w), name
    assert plan.workspace.status() == 0


@pytest.mark.parametrize("kind", ["process", "distill"])
def test_run_on_several_streams_in_turn(kind):
    z, ids, logq = teacher(60, 5003, 8, 4)
    if kind == "process":
        plan = ds.ProcessPlan(z.view(20, 3, -1), **request(20, 3, 5003, 300, 40, 5))
        first = lambda: plan.out
    else:
        plan = ds.DistillPlan(z, ids, logq)
        first = lambda: plan.out.grad_logits
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


@pytest.mark.parametrize("B,R,V", [(90, 2, 30011), (700, 1, 9001), (160, 5, 2048)])
def test_requests_together_and_one_by_one(B, R, V):
    """How a call's vocabulary is sliced depends on B; its results do not."""
    r = request(B, R, V, 700, 70, 6)
    z = torch.randn(B, R, V, device="cuda")
    y = ds.process_logits(z, **r)
    g = ds.process_logits_grad(z.flip(0), z, **{k: r[k] for k in ("history", "drafted", "repetition", "mask", "mask_rows")})
    for b in (0, 1, B // 2, B - 1):
        one = {k: v if k == "mask" else v[b:b + 1] for k, v in r.items()}
        assert torch.equal(ds.process_logits(z[b:b + 1], **one), y[b:b + 1])
        one = {k: one[k] for k in ("history", "drafted", "repetition", "mask", "mask_rows")}
        assert torch.equal(ds.process_logits_grad(z.flip(0)[b:b + 1], z[b:b + 1], **one), g[b:b + 1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,pad", [(17000, 130, 0), (700, 50021, 3)])
def test_the_loss_alone_in_calls_of_any_size(N, V, pad, dtype):
    """Few rows' losses take one launch and many rows' two; a row's bits are the same."""
    K = 5
    g = torch.Generator(device="cuda").manual_seed(7)
    z = (torch.randn(N, V + pad, generator=g, device="cuda") * 3).to(dtype)[:, :V]
    ids = torch.randint(0, V // K, (N, K), generator=g, device="cuda") + torch.arange(K, device="cuda") * (V // K)
    ids = ids.to(torch.int32)
    logq = torch.log(torch.rand(N, K, generator=g, device="cuda") / K)
    big = ds.distill_loss(z, ids, logq, alpha=(0.3, 0.7), want_grad=False)
    assert big.grad_logits is None
    for i, j in ((0, 1), (N // 2, N // 2 + 7), (N - 3, N)):
        few = ds.distill_loss(z[i:j], ids[i:j], logq[i:j], alpha=(0.3, 0.7), want_grad=False)
        for name in ("loss", "parts", "norm"):
            assert torch.equal(getattr(few, name), getattr(big, name)[i:j]), name


@pytest.mark.parametrize("N,V", [(6, 3000), (17000, 130), (3, 1_700_000)])
@pytest.mark.parametrize("grad", [True, False])
def test_padding_rows_may_hold_anything(N, V, grad):
    """One launch and several: rows of weight 0, with NaN logits and impossible ids, give 0 and set no status."""
    z, ids, logq = teacher(N, V, 4, 8)
    w = torch.ones(N, device="cuda")
    want = ds.distill_loss(z, ids, logq, weight=w, want_grad=grad)
    w[1] = 0.0
    z[1], ids[1], logq[1] = float("nan"), V + 5, float("nan")
    ws = ds.DistillWorkspace(N, V, 4)
    o = ds.distill_loss(z, ids, logq, weight=w, want_grad=grad, workspace=ws)
    assert ws.status() == 0
    for name in ("loss", "parts", "norm") + (("grad_logits",) if grad else ()):
        x, y = getattr(o, name), getattr(want, name)
        assert not x[1].any() and torch.equal(x[0], y[0]) and torch.equal(x[2:], y[2:]), name
    if grad:
        g = ds.distill_grad(z, ids, logq, o.norm, w, workspace=ws)
        assert ws.status() == 0 and not g[1].any() and torch.isfinite(g).all()
