"""Table rows for given tokens (exact) and the table's gradient against plain 64-bit forms.

A row's gradient is a sum of n fp32 terms: any order is off by at most n 2^-24 sum |terms|; the scale
and a bf16 result add one rounding each."""
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

DT = [torch.float32, torch.bfloat16]


def tokens(N, V, seed, kind="mixed"):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    if kind == "one":
        t[:] = V - 1
    elif kind == "text":        # frequencies fall as 1 / rank
        t = (torch.rand(N, generator=g, dtype=torch.float64) * torch.log(torch.tensor(V + 1.0))).exp()
        t = (t - 1).long().clamp(0, V - 1).to(torch.int32)
    elif kind == "distinct":
        t = torch.randperm(V, generator=g)[:N].to(torch.int32)
    elif kind == "ascending":
        t = torch.sort(t).values
    if kind == "mixed" and N > 4:
        t[::5] = -1
        t[1], t[2] = 0, V - 1
    return t


@pytest.mark.gpu
@pytest.mark.parametrize("wdt", DT)
@pytest.mark.parametrize("odt", DT)
@pytest.mark.parametrize("N,V,D,scale", [(1, 1, 1, 1.0), (7, 50, 3, 2.0), (100, 1000, 64, 0.5), (33, 77, 250, 1.0),
                                         (9, 100, 1023, 3.0), (5, 60, 4096, 64.0), (1000, 333, 256, 1.0),
                                         (3, 9, 20000, 0.1)])
def test_embedding(N, V, D, scale, wdt, odt):
    g = torch.Generator().manual_seed(N + V + D)
    W = torch.randn(V, D, generator=g).to(wdt)
    t = tokens(N, V, 3)
    got = ds.embedding(W.cuda(), t.cuda(), scale=scale, dtype=odt).cpu()
    want = (W[t.long().clamp(min=0)].float() * scale).to(odt)
    want[t < 0] = 0
    assert got.dtype == odt and torch.equal(got, want)


@pytest.mark.gpu
def test_embedding_shapes_and_invalid_tokens():
    W = torch.randn(50, 16).cuda()
    t = tokens(12, 50, 4).view(3, 4).cuda()
    assert ds.embedding(W, t).shape == (3, 4, 16)
    assert ds.embedding(W, torch.empty(0, dtype=torch.int32, device="cuda")).shape == (0, 16)
    bad = torch.tensor([3, 50, -2, -1, 7], dtype=torch.int32, device="cuda")
    o = ds.embedding(W, bad)
    assert torch.isnan(o[1]).all() and torch.isnan(o[2]).all() and (o[3] == 0).all()
    assert torch.equal(o[[0, 4]], W[[3, 7]])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DT)
def test_embedding_views(dt):
    # table and output that start anywhere in a buffer
    buf = torch.randn(40 * 64 + 8).to(dt).cuda()
    t = tokens(20, 40, 5).cuda()
    for off in (1, 2, 3, 4):
        W = buf[off:off + 40 * 64].view(40, 64)
        out = torch.empty(20 * 64 + 8, dtype=dt, device="cuda")[off - 1:][:20 * 64].view(20, 64)
        ds.embedding(W, t, out=out)
        want = W[t.long().clamp(min=0)].clone()
        want[t < 0] = 0
        assert torch.equal(out, want)


@pytest.mark.gpu
def test_embedding_past_32_bit_offsets():
    V, D = 140000, 40000
    W = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    W[-3:].normal_()
    t = torch.tensor([V - 1, V - 3], dtype=torch.int32, device="cuda")
    assert torch.equal(ds.embedding(W, t), W[[V - 1, V - 3]])


# ------------------------------------------------------------------ gradient
def reference_grad(g, t, V, scale):
    out = torch.zeros(V, g.shape[1], dtype=torch.float64)
    size = torch.zeros_like(out)
    keep = (t >= 0) & (t < V)
    for i in keep.nonzero()[:, 0].tolist():
        out[t[i]] += g[i].double()
        size[t[i]] += g[i].double().abs()
    n = torch.bincount(t[keep].long(), minlength=V).double()[:, None]
    return out * scale, size * abs(scale), n


def check_grad(g, t, V, scale=1.0, odt=torch.float32, base=None, ws=None):
    out = None if base is None else base.cuda()
    ws = ws or ds.EmbeddingGradWorkspace(t.numel(), V, g.shape[1])
    got = ds.embedding_grad(g.cuda(), t.cuda(), V, scale=scale, dtype=odt, accumulate=base is not None,
                            out=out, workspace=ws)
    torch.cuda.synchronize()
    assert ws.status() == 0
    want, size, n = reference_grad(g, t, V, scale)
    tol = (n + 2) * 2.0 ** -24 * size
    if base is not None:
        want = want + base.double()
        tol = tol + 2.0 ** -23 * (size + base.double().abs()) * (n > 0)
    if odt == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    err = (got.double().cpu() - want).abs()
    assert got.dtype == odt and (err <= tol).all(), float((err - tol).max())
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("gdt", DT)
@pytest.mark.parametrize("N,V,D,kind", [(1, 1, 1, "one"), (1, 5, 8, "one"), (2, 3, 250, "one"), (33, 10, 64, "mixed"),
                                        (448, 3000, 256, "text"), (512, 2, 31, "mixed"), (700, 100000, 8, "mixed"),
                                        (1000, 500, 130, "one"), (2000, 4001, 64, "distinct"),
                                        (3584, 900, 72, "ascending"), (5000, 1000, 33, "text"),
                                        (20000, 5000, 16, "text"), (9000, 70000, 12, "one")])
def test_embedding_grad(N, V, D, kind, gdt):
    g = torch.randn(N, D, generator=torch.Generator().manual_seed(N + D)).to(gdt)
    check_grad(g, tokens(N, V, N, kind), V, scale=1.0 if D % 2 else 0.75)


@pytest.mark.gpu
@pytest.mark.parametrize("N,V,D", [(50, 40, 24), (6000, 300, 20)])
def test_embedding_grad_bf16_and_accumulate(N, V, D):
    g = torch.randn(N, D, generator=torch.Generator().manual_seed(7))
    t = tokens(N, V, 8)
    check_grad(g, t, V, odt=torch.bfloat16)
    check_grad(g.bfloat16(), t, V, scale=2.0, odt=torch.bfloat16)
    base = torch.randn(V, D, generator=torch.Generator().manual_seed(9))
    check_grad(g, t, V, base=base)
    check_grad(g, t, V, odt=torch.bfloat16, base=base.bfloat16())
    # rows of absent tokens keep their bits, NaN among them
    absent = torch.full((V + 3, D), float("nan"))
    absent[:V] = base
    got = check_grad(g, t, V, base=base)
    out = absent.cuda()
    ds.embedding_grad(g.cuda(), t.cuda(), V + 3, accumulate=True, out=out)
    assert torch.equal(out[:V], got) and torch.isnan(out[V:]).all()


@pytest.mark.gpu
def test_embedding_grad_order_and_workspace_reuse():
    # the same call twice gives the same bits, and one workspace serves smaller problems too
    ws = ds.EmbeddingGradWorkspace(9000, 5000, 40)
    for N, V, D, kind in [(9000, 5000, 40, "text"), (100, 60, 40, "mixed"), (9000, 5000, 40, "text"),
                          (4000, 10, 8, "mixed")]:
        g = torch.randn(N, D, generator=torch.Generator().manual_seed(N)).cuda()
        t = tokens(N, V, 10, kind).cuda()
        a = ds.embedding_grad(g, t, V, workspace=ws)
        b = ds.embedding_grad(g, t, V, workspace=ws)
        c = ds.embedding_grad(g, t, V)
        assert torch.equal(a, b) and torch.equal(a, c)
        assert ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N", [500, 9000])
def test_embedding_grad_in_a_graph(N):
    V, D = 3000, 72
    g = torch.randn(N, D, generator=torch.Generator().manual_seed(N)).cuda()
    plan = ds.EmbeddingGradPlan(g, tokens(N, V, 11, "text").cuda(), V)
    plan.run()
    torch.cuda.synchronize()
    want = plan.out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(torch.cuda.current_stream())
    for _ in range(3):
        plan.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(plan.out, want)


@pytest.mark.gpu
def test_embedding_grad_no_tokens_and_all_padding():
    out = ds.embedding_grad(torch.empty(0, 12, device="cuda"),
                            torch.empty(0, dtype=torch.int32, device="cuda"), 30)
    assert (out == 0).all() and out.shape == (30, 12)
    t = torch.full((70,), -1, dtype=torch.int32, device="cuda")
    assert (ds.embedding_grad(torch.ones(70, 12, device="cuda"), t, 30) == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [60, 9000])
def test_embedding_grad_invalid_tokens(N):
    g = torch.randn(N, 16).cuda()
    t = tokens(N, 40, 12)
    u = t.clone()
    u[3], u[7] = 40, -9
    t[3] = t[7] = -1
    ws = ds.EmbeddingGradWorkspace(N, 40, 16)
    got = ds.embedding_grad(g, u.cuda(), 40, workspace=ws)
    assert ws.status() == 1 and ws.status() == 0
    assert torch.equal(got, ds.embedding_grad(g, t.cuda(), 40, workspace=ws))


@pytest.mark.gpu
def test_embedding_grad_other_stream_and_views():
    N, V, D = 300, 90, 48
    buf = torch.randn(N * D + 3).cuda()
    t = tokens(N, V, 13).cuda()
    g = buf[3:].view(N, D)
    want = ds.embedding_grad(g.clone(), t, V)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty(V * D + 1, device="cuda")[1:].view(V, D)
    s.wait_stream(torch.cuda.current_stream())
    ds.embedding_grad(g, t, V, stream=s, out=out)
    s.synchronize()
    assert torch.equal(out, want)


@pytest.mark.gpu
def test_embedding_against_differences():
    """d/dW of a linear functional of the looked-up rows is the gradient call's result."""
    V, D, N = 6, 4, 9
    g = torch.Generator().manual_seed(14)
    W, dy = torch.randn(V, D, generator=g).cuda(), torch.randn(N, D, generator=g).cuda()
    t = tokens(N, V, 15).cuda()
    grad = ds.embedding_grad(dy, t, V, scale=1.5)
    for v in range(V):
        for j in range(D):
            up, dn = W.clone(), W.clone()
            up[v, j] += 0.5
            dn[v, j] -= 0.5
            diff = ((ds.embedding(up, t, scale=1.5).double() - ds.embedding(dn, t, scale=1.5).double())
                    * dy.double()).sum()
            assert abs(float(diff - grad[v, j])) < 1e-5


@pytest.mark.gpu
def test_refusals():
    W = torch.randn(10, 8).cuda()
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        ds.embedding(W.cpu(), t)
    with pytest.raises(TypeError):
        ds.embedding(W.double(), t)
    with pytest.raises(TypeError):
        ds.embedding(W, t.long())
    with pytest.raises(ValueError):
        ds.embedding(W[:, :4], t)
    with pytest.raises(ValueError):
        ds.embedding(W, t, out=torch.empty(4, 7, device="cuda"))
    with pytest.raises(ds._lib.DsparkError):
        ds.embedding(W, t, scale=float("nan"))
    g = torch.randn(4, 8).cuda()
    with pytest.raises(ValueError):
        ds.embedding_grad(g[:3], t, 10)
    with pytest.raises(ValueError):
        ds.embedding_grad(g, t, 10, accumulate=True)
    with pytest.raises(ValueError):
        ds.embedding_grad(g, t, 10, out=torch.empty(9, 8, device="cuda"))
    with pytest.raises(ds._lib.DsparkError):
        ws = ds.EmbeddingGradWorkspace(4, 10, 8)
        ws.nbytes = 64
        ds.embedding_grad(g, t, 10, workspace=ws)
