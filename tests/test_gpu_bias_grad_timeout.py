"""The bias gradients' timeout path, exercised without faulting or hanging the GPU.

The test hook DSPARK_TEST_STUCK_WAIT (read at every call) makes a wait run out after 20 us: mbar, that of
the warps that read the accumulators; mma, that of the thread that issues the MMAs.  The other roles of the
block, and of a pair's other block, see it and stop; copies and MMAs in flight end; TMEM is freed.  The call
reports DSPARK_ERR_TIMEOUT, and the next one on the same workspace is right."""
import time

import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wait", ["mbar", "mma"])
# pairs, a split fp32 gradient by TMA, fp32 and bf16 rows brought by warps; short and long sums, both layouts
@pytest.mark.parametrize("gdt,N,V,r,layout", [(torch.bfloat16, 300, 40000, 128, "vr"), (torch.bfloat16, 40, 512, 8, "rv"),
                                              (torch.float32, 300, 40000, 128, "vr"), (torch.float32, 40, 512, 72, "rv"),
                                              (torch.float32, 70, 9001, 128, "vr"), (torch.bfloat16, 70, 9001, 128, "vr")])
def test_a_wait_that_runs_out(monkeypatch, wait, gdt, N, V, r, layout):
    g = torch.Generator(device="cuda").manual_seed(N + V)
    G = torch.randn(N, V, generator=g, device="cuda").to(gdt)
    a = torch.randn(N, r, generator=g, device="cuda").bfloat16()
    W2 = torch.randn(*((V, r) if layout == "vr" else (r, V)), generator=g, device="cuda").bfloat16()
    plan = ds.BiasGradPlan(G, a, W2, w2_layout=layout)
    plan.run()
    assert plan.workspace.status() == 0
    want = [x.clone() for x in plan.out]
    monkeypatch.setenv("DSPARK_TEST_STUCK_WAIT", wait)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    plan.run()
    status = plan.workspace.status()
    elapsed = time.perf_counter() - t0
    assert status == 4, status
    # two products, in each at most a block's waits for copies that the pair's other block never began and
    # for signals of stages that were never reached: one limit of a second each
    assert elapsed < 8.0, elapsed
    monkeypatch.delenv("DSPARK_TEST_STUCK_WAIT")
    for x in plan.out:
        x.fill_(float("nan"))
    plan.run()
    assert plan.workspace.status() == 0
    assert all(torch.equal(x, y) for x, y in zip(plan.out, want))
    print(f"{wait} {gdt}: ended in {elapsed * 1e3:.1f} ms")
