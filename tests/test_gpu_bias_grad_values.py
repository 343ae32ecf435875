"""Gradients of the bias product from bf16 tables, held to the arithmetic that the kernel implements.

Every product of two bf16 numbers is exact in fp32, and an fp32 gradient enters as three bf16 parts
that hold all its bits.  What is left: an addition into an accumulator drops at most one unit in its
last place, 2^-23 of it, and a run of at most 32 additions ends in an fp32 sum rounded to nearest.  A
run's accumulator is about sqrt(squares of its terms), and the runs' squares add up to s^2 for
s = sqrt(squares of all terms).  So the error of all elements together, against their s together, is
at most about (32 + sqrt(runs)) 2^-23; the accumulated result adds a rounding."""
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

BF = torch.bfloat16


def inputs(N, V, r, gdt, layout, seed):
    g = torch.Generator().manual_seed(seed)
    G = (torch.randn(N, V, generator=g) * 0.1).to(gdt)
    a = torch.randn(N, r, generator=g).to(BF)
    W2 = torch.randn(*((V, r) if layout == "vr" else (r, V)), generator=g).to(BF)
    return G, a, W2


def norm_error(got, A, B):
    """|got - A B| over all elements, against the root of their terms' squares."""
    A, B = A.double().cuda(), B.double().cuda()
    return float((got.double() - A @ B).norm() / ((A * A) @ (B * B)).sum().sqrt())


def bound(K):
    return (32 + (K / 512 + 1) ** 0.5) * 2.0 ** -23


def check(N, V, r, gdt, layout):
    G, a, W2 = inputs(N, V, r, gdt, layout, N + V + r)
    ws = ds.BiasGradWorkspace(N, V, r)
    ga, gw = ds.bias_grad(G.cuda(), a.cuda(), W2.cuda(), w2_layout=layout, workspace=ws)
    torch.cuda.synchronize()
    assert ws.status() == 0
    W = W2.t() if layout == "rv" else W2
    gw = gw.t() if layout == "rv" else gw
    ea, ew = norm_error(ga, G, W), norm_error(gw, G.t(), a)
    assert ea <= bound(V) and ew <= bound(N), (ea, bound(V), ew, bound(N))


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["vr", "rv"])
@pytest.mark.parametrize("N,V,r", [(1, 8, 8), (300, 4096, 8), (70, 2056, 16), (129, 5000, 24), (513, 8192, 72),
                                   (256, 3000, 80), (40, 1024, 200), (300, 2048, 264), (31, 4000, 272)])
def test_pair_of_any_rank(N, V, r, layout):
    # bf16 rows of a multiple of 16 bytes, ranks that fill the last columns of a tile in part
    check(N, V, r, BF, layout)


def same_kind(got, want, tol):
    """NaN where the 64-bit product has NaN, its infinities with their signs, and near it elsewhere."""
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])
    on = torch.isfinite(want)
    assert ((got - want)[on].abs() <= tol * want[on].abs().clamp(min=1.0)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("gdt", [torch.float32, BF])
@pytest.mark.parametrize("V", [3000, 3001, 3002])    # every way in which rows are brought
def test_infinities_nan_and_the_largest_numbers(V, gdt):
    inf, top = float("inf"), torch.finfo(gdt).max
    G, a, W2 = inputs(40, V, 64, gdt, "vr", 5)
    G[3, 1234], G[5, 70], G[5, 71], G[9, 77] = inf, -inf, inf, float("nan")
    ga, gw = ds.bias_grad(G.cuda(), a.cuda(), W2.cuda())
    same_kind(ga, G.double() @ W2.double(), 1e-3)     # (sums of some thousand terms of 0.1)
    same_kind(gw, G.double().t() @ a.double(), 1e-3)

    # the largest numbers, alone in their rows and columns, with factors that keep the products finite
    big = torch.zeros(40, V).to(gdt)
    big[2, 0], big[7, 129], big[39, V - 1] = top, -top, top
    if gdt == torch.float32:
        big[20, 500] = 3.3953e38                      # above bf16's largest number
    a, W2 = (a.float().clamp(-0.9, 0.9)).to(BF), (W2.float().clamp(-0.9, 0.9)).to(BF)
    ga, gw = ds.bias_grad(big.cuda(), a.cuda(), W2.cuda())
    same_kind(ga, big.double() @ W2.double(), 2.0 ** -20)
    same_kind(gw, big.double().t() @ a.double(), 2.0 ** -20)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["vr", "rv"])
@pytest.mark.parametrize("gdt", [torch.float32, BF])
@pytest.mark.parametrize("N,V,r", [(200, 40000, 64), (64, 20002, 256), (3000, 1000, 72), (2500, 515, 264)])
def test_long_sums(N, V, r, gdt, layout):
    # accumulators that were never emptied would be 1e-5 off, two parts of an fp32 gradient 3e-6 or more
    check(N, V, r, gdt, layout)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [4096, 4097])
def test_the_last_bits_of_an_fp32_gradient(V):
    """Entries 1 + k 2^-23 against entries 1 with the opposite factor: only the last eight bits are left.
    The factors have six bits, so every sum of the upper parts is exact and cancels; without the third
    part the result is zero."""
    g = torch.Generator().manual_seed(9)
    N, r = 96, 64
    k = torch.randint(1, 256, (N, V), generator=g)
    k[:, 1::2] = 0
    G = 1.0 + k.float() * 2.0 ** -23
    if V % 2:
        G[:, -1] = 0.0
    w = (32 + torch.randint(0, 32, (V // 2, r), generator=g)).float() / 32
    W2 = torch.zeros(V, r)
    W2[0:V - V % 2:2], W2[1:V:2] = w, -w
    a = torch.zeros(N, r)
    h = (32 + torch.randint(0, 32, (N // 2, r), generator=g)).float() / 32
    a[0::2], a[1::2] = h, -h
    ga, _ = ds.bias_grad(G.cuda(), a.to(BF).cuda(), W2.to(BF).cuda())
    H = 1.0 + torch.randint(1, 256, (N, V), generator=g).float() * 2.0 ** -23
    H[1::2] = 1.0
    _, gw = ds.bias_grad(H.cuda(), a.to(BF).cuda(), W2.to(BF).cuda())
    for got, want in ((ga, G.double() @ W2.double()), (gw, H.double().t() @ a.double())):
        assert ((got.double().cpu() - want).abs() <= 2.0 ** -10 * want.abs()).all()
        assert (want.abs() > 0).all()
