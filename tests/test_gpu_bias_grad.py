"""Gradients of the bias product a W2 against 64-bit products.

A sum of K fp32 terms whose partial sums stay near s = sqrt(sum of squared terms) is off by at most
about K 2^-24 of a few s; reading fp32 gradients of the logits to 16 significant bits or more adds
2^-16 s.  The bound below, (K 2^-24 + 2^-15) 4 s, is still far below one missing term, about
s / sqrt(K)."""
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds


def make(N, V, r, gdt, wdt, layout, seed):
    g = torch.Generator().manual_seed(seed)
    G = (torch.randn(N, V, generator=g) * 0.1).to(gdt)
    a = torch.randn(N, r, generator=g).to(wdt)
    W2 = torch.randn(*((V, r) if layout == "vr" else (r, V)), generator=g).to(wdt)
    return G, a, W2


def bound(A, B, K):
    return 4 * (K * 2.0 ** -24 + 2.0 ** -15) * ((A * A) @ (B * B)).sqrt() + 1e-30


def check(N, V, r, gdt, wdt, layout, seed=0, accumulate=False):
    G, a, W2 = make(N, V, r, gdt, wdt, layout, seed + N + V + r)
    ws = ds.BiasGradWorkspace(N, V, r, wdt == torch.bfloat16)
    out = None
    base = torch.zeros(W2.shape)
    if accumulate:
        base = torch.randn(W2.shape, generator=torch.Generator().manual_seed(1))
        out = (torch.full((N, r), float("nan"), device="cuda"), base.cuda())
    for _ in range(1 if accumulate else 2):
        ga, gw = ds.bias_grad(G.cuda(), a.cuda(), W2.cuda(), w2_layout=layout, workspace=ws, out=out,
                              accumulate=accumulate)
    torch.cuda.synchronize()
    assert ws.status() == 0
    Gd, ad, Wd = G.double(), a.double(), W2.double()
    if layout == "rv":
        Wd, gw, base = Wd.t(), gw.t(), base.t()
    ea = (ga.double().cpu() - Gd @ Wd).abs()
    ew = (gw.double().cpu() - (Gd.t() @ ad + base.double())).abs()
    assert (ea <= bound(Gd, Wd, V)).all(), float(ea.max())
    assert (ew <= bound(Gd.t(), ad, N) + 2.0 ** -22 * base.double().abs()).all(), float(ew.max())


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["vr", "rv"])
@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("wdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,r", [(1, 2, 8), (28, 4096, 64), (5, 1001, 72), (130, 333, 16)])
def test_bias_grad_small(N, V, r, gdt, wdt, layout):
    check(N, V, r, gdt, wdt, layout)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["vr", "rv"])
@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,r", [(1, 5000, 256), (7, 20000, 256), (448, 12345, 256), (129, 8192, 64),
                                   (128, 8200, 200), (300, 3001, 512), (64, 40000, 320), (700, 2056, 128)])
def test_bias_grad_bf16_weights(N, V, r, gdt, layout):
    check(N, V, r, gdt, torch.bfloat16, layout)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["vr", "rv"])
@pytest.mark.parametrize("gdt,wdt", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16),
                                     (torch.float32, torch.float32)])
def test_bias_grad_accumulates(gdt, wdt, layout):
    check(100, 3000, 64, gdt, wdt, layout, accumulate=True)


@pytest.mark.gpu
def test_bias_grad_shapes_and_no_rows():
    G, a, W2 = make(12, 500, 64, torch.float32, torch.bfloat16, "vr", 3)
    ga, gw = ds.bias_grad(G.cuda(), a.cuda(), W2.cuda())
    gb, gx = ds.bias_grad(G.cuda().view(3, 4, 500), a.cuda().view(3, 4, 64), W2.cuda())
    assert gb.shape == (3, 4, 64) and torch.equal(gb.view(12, 64), ga) and torch.equal(gw, gx)
    ga, gw = ds.bias_grad(G[:0].cuda(), a[:0].cuda(), W2.cuda())
    assert ga.shape == (0, 64) and (gw == 0).all()


@pytest.mark.gpu
def test_bias_grad_repeat_identical_and_other_stream():
    G, a, W2 = [x.cuda() for x in make(200, 30000, 256, torch.float32, torch.bfloat16, "vr", 4)]
    x = ds.bias_grad(G, a, W2)
    y = ds.bias_grad(G, a, W2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = ds.bias_grad(G, a, W2, stream=s)
    s.synchronize()
    for p in (y, z):
        assert torch.equal(x[0], p[0]) and torch.equal(x[1], p[1])


@pytest.mark.gpu
@pytest.mark.parametrize("gdt,V", [(torch.float32, 4096), (torch.bfloat16, 4096), (torch.bfloat16, 4099)])
def test_bias_grad_in_a_graph(gdt, V):
    G, a, W2 = [x.cuda() for x in make(300, V, 128, gdt, torch.bfloat16, "vr", 8)]
    plan = ds.BiasGradPlan(G, a, W2)
    plan.run()
    torch.cuda.synchronize()
    want = [x.clone() for x in plan.out]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run(torch.cuda.current_stream())
    for _ in range(3):
        for x in plan.out:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(plan.out, want))
    assert plan.workspace.status() == 0


@pytest.mark.gpu
def test_bias_grad_keeps_infinities_and_nan():
    # what is not finite reaches the rows that it touches and no others
    G, a, W2 = make(40, 3000, 64, torch.float32, torch.bfloat16, "vr", 5)
    G[7, 1234] = float("inf")
    G[9, 77] = float("nan")
    ga, gw = ds.bias_grad(G.cuda(), a.cuda(), W2.cuda())
    bad_a, bad_w = ~torch.isfinite(ga).all(1).cpu(), ~torch.isfinite(gw).all(1).cpu()
    assert bad_a.nonzero()[:, 0].tolist() == [7, 9] and bad_w.nonzero()[:, 0].tolist() == [77, 1234]


@pytest.mark.gpu
def test_bias_grad_against_differences():
    """The gradients of L = sum G * (a W2^T): L is linear in either factor, so a difference of one
    whole unit is exact up to rounding."""
    G, a, W2 = make(3, 16, 8, torch.float32, torch.float32, "vr", 6)
    ga, gw = ds.bias_grad(G.cuda(), a.cuda(), W2.cuda())
    L = lambda p, q: (G.double() * (p.double() @ q.double().t())).sum()
    for n, j in [(0, 0), (2, 7), (1, 3)]:
        p = a.clone().double()
        p[n, j] += 1.0
        assert abs(float(L(p, W2) - L(a, W2)) - float(ga[n, j])) < 1e-5
    for v, j in [(0, 0), (15, 7), (9, 2)]:
        q = W2.clone().double()
        q[v, j] += 1.0
        assert abs(float(L(a, q) - L(a, W2)) - float(gw[v, j])) < 1e-5


@pytest.mark.gpu
def test_refusals():
    G, a, W2 = [x.cuda() for x in make(4, 100, 16, torch.float32, torch.bfloat16, "vr", 7)]
    with pytest.raises(ValueError):
        ds.bias_grad(G.cpu(), a, W2)
    with pytest.raises(TypeError):
        ds.bias_grad(G, a.float(), W2)
    with pytest.raises(ValueError):
        ds.bias_grad(G, a, W2, w2_layout="rv")
    with pytest.raises(ValueError):
        ds.bias_grad(G, a[:3], W2)
    with pytest.raises(ValueError):
        ds.bias_grad(G, a, W2, accumulate=True)
    with pytest.raises(ValueError):
        ds.bias_grad(G[:, ::2], a, W2[:50])
    with pytest.raises((ValueError, ds._lib.DsparkError)):   # r not a multiple of 8
        ds.bias_grad(G, a[:, :12].contiguous(), W2[:, :12].contiguous())
    with pytest.raises(ds._lib.DsparkError):                  # 16-byte alignment
        ds.bias_grad(torch.randn(401, device="cuda")[1:].view(4, 100), a, W2)
