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
