"""Distillation from a teacher's largest log probabilities, and its gradient, against plain 64-bit forms.

Tolerances, from the arithmetic: an exponential in fp32 is off by about 2^-22 + |d| 2^-23 of itself (d = (z -
max) / T), so a sum's logarithm is off by at most e = 2^-21 (1 + E|d|), of the row and of the rest alike (e_r).
The outcomes are formed to less than that from pairs of fp32 numbers: ln p_j is off by e, ln p_r by e + e_r, and KL,
L1 and M by at most e + e_r times the sum of the probabilities they weigh (KL: the teacher's, 1; L1 and M: the
student's, 1), twice for both.  P_v is off by 2^-21 (4 + |ln P_v|) of itself, and bf16 results by 2^-8."""
import math

import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

EPS = 2.0 ** -21
U = 2.0 ** -24


def sums(z, T):
    """(maximum, ln sum, E|d|) of a row in float64; a row that is -inf everywhere: (-inf, 0, 0)."""
    some = z > -math.inf
    if not some.any():
        return -math.inf, 0.0, 0.0
    m = z.max()
    d = torch.where(some, (z - m) / T, torch.zeros_like(z))
    e = torch.where(some, torch.exp(d), torch.zeros_like(z))
    return float(m), float(e.sum().log()), float((e * d.abs()).sum() / e.sum())


def reference(z, ids, lq, T, alpha, rest, w):
    """Row by row in float64: dict of loss, parts, norm, grad and their bounds."""
    N, V = z.shape
    r = dict(loss=torch.zeros(N), parts=torch.zeros(N, 2), norm=torch.zeros(N, 4), grad=torch.zeros(N, V),
             tloss=torch.zeros(N), tparts=torch.zeros(N), tnorm=torch.zeros(N, 4), tgrad=torch.zeros(N, V))
    r = {k: v.double() for k, v in r.items()}
    a, b = alpha
    for i in range(N):
        if w[i] == 0:
            continue
        row, S = z[i].double(), [(int(t), float(l)) for t, l in zip(ids[i], lq[i]) if t >= 0]
        out = row.clone()
        out[[t for t, _ in S]] = -math.inf
        m, ls, ed = sums(row, T)
        mr, lsr, edr = sums(out, T)
        e, er = EPS * (1 + ed), EPS * (1 + edr)
        none = m == -math.inf
        lnp = lambda x: -math.inf if x == -math.inf or none else (x - m) / T - ls
        lpr = -math.inf if mr == -math.inf else (mr - m) / T + lsr - ls
        q = [math.exp(l) for _, l in S]
        p = [math.exp(lnp(float(row[t]))) for t, _ in S]
        qr, pr = max(0.0, 1.0 - sum(q)), math.exp(lpr)
        kl = sum(qq * (l - lnp(float(row[t]))) for qq, (t, l) in zip(q, S) if qq > 0)
        l1 = sum(abs(x - y) for x, y in zip(p, q))
        if rest:
            kl += qr * (math.log(qr) - lpr) if qr > 0 else 0.0
            l1 += abs(pr - qr)
        r["parts"][i, 0], r["parts"][i, 1] = kl, l1
        r["loss"][i] = float(w[i]) * ((a * kl if a else 0.0) + (b * l1 if b else 0.0))
        r["norm"][i] = torch.tensor([m, ls, mr, lsr], dtype=torch.float64)
        r["tnorm"][i] = torch.tensor([0.0, e + er, 0.0, er], dtype=torch.float64)
        off = 2 * (e + er)
        r["tparts"][i] = off
        r["tloss"][i] = abs(float(w[i])) * (abs(a) + abs(b)) * off
        sgn = lambda x: (x > 0) - (x < 0)
        t = [-a * y + b * x * sgn(x - y) for x, y in zip(p, q)]
        tr = -a * qr + b * pr * sgn(pr - qr) if rest else 0.0
        M = sum(t) + tr
        dM = abs(b) * off
        s = float(w[i]) / T
        if mr > -math.inf:
            lnP = torch.where(out > -math.inf, (out - mr) / T - lsr, torch.full_like(out, -math.inf))
            P = lnP.exp()
            c = s * (tr - pr * M)
            dc = abs(s) * pr * ((abs(b) + abs(M)) * (e + er) + dM)
            r["grad"][i] = c * P
            lim = torch.where(P > 0, lnP.abs(), torch.zeros_like(P))
            r["tgrad"][i] = P * (abs(c) * EPS * (4 + lim) + dc) + 2.0 ** -126
        for (tok, _), x, tt in zip(S, p, t):
            r["grad"][i, tok] = s * (tt - x * M)
            r["tgrad"][i, tok] = abs(s) * x * ((abs(b) + abs(M)) * e + dM)
    return r


def close(name, got, want, tol):
    got, want = got.double().cpu(), want.double()
    tol = tol.expand_as(want) + U * torch.where(torch.isfinite(want), want.abs(), torch.zeros_like(want))
    assert torch.equal(torch.isnan(got), torch.isnan(want)), name
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), name
    fine = torch.isfinite(want)
    err = (got - want)[fine].abs()
    assert (err <= tol[fine]).all(), (name, float((err - tol[fine]).max()), float(err.max()))


def check(z, ids, lq, T=1.0, alpha=(1.0, 0.0), rest=True, weight=None, zc=None):
    zc = z.cuda() if zc is None else zc
    N, V = z.shape
    K = ids.shape[1]
    w = torch.ones(N) if weight is None else weight
    want = reference(z.float(), ids, lq, T, alpha, rest, w)
    ws = ds.DistillWorkspace(N, V, K)
    kw = dict(T=T, alpha=alpha, rest=rest)
    wc = None if weight is None else weight.cuda()
    for _ in range(2):  # the second call meets the workspace as the first one left it
        o = ds.distill_loss(zc, ids.cuda(), lq.cuda(), weight=wc, workspace=ws, **kw)
    f = ds.distill_loss(zc, ids.cuda(), lq.cuda(), weight=wc, want_grad=False, workspace=ws, **kw)
    g = ds.distill_grad(zc, ids.cuda(), lq.cuda(), o.norm, w.cuda(), workspace=ws, **kw)
    assert ws.status() == 0 and f.grad_logits is None
    rnd = 2.0 ** -8 if z.dtype == torch.bfloat16 else 0.0
    for x in (o, f):
        close("loss", x.loss, want["loss"], want["tloss"])
        close("parts", x.parts, want["parts"], want["tparts"][:, None])
        close("norm", x.norm, want["norm"], want["tnorm"])
    for x in (o.grad_logits, g):
        # (from norms rounded to fp32: half a step of each logarithm more)
        more = 1 + 4 * rnd
        close("grad", x, want["grad"], want["tgrad"] * more + rnd * want["grad"].abs()
              + U * want["grad"].abs() * (2 + want["norm"][:, 1:2].abs() + want["norm"][:, 3:].abs()))
    return o


def make(N, V, K, seed, dtype=torch.float32, std=3.0, pad=True):
    """Logits, and a teacher whose K tokens the student has near its own probabilities."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, V, generator=g) * std
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)]).to(torch.int32)
    q = torch.rand(N, K, generator=g) ** 4 + 1e-4
    q = q / q.sum(1, keepdim=True) * (0.5 + 0.45 * torch.rand(N, 1, generator=g))
    lift = math.log(V) + std * std / 2 + (q.log() + torch.randn(N, K, generator=g))
    if K < V:
        z.scatter_(1, ids.long(), lift)
    lq = q.log()
    if pad and K > 2:
        ids[0, K - 2:], lq[0, K - 2:] = -1, -math.inf
    return z.to(dtype), ids, lq


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("N,V,K", [(1, 2, 1), (1, 2, 2), (2, 3, 2), (3, 31, 5), (2, 128, 128), (5, 1001, 7),
                                   (4, 4096, 32), (3, 8191, 128), (2, 8193, 20), (7, 16384, 1), (1, 50021, 64),
                                   (2, 151936, 50), (40, 1000, 33), (1, 262144, 128), (160, 3000, 6)])
def test_distill(N, V, K, rest, dtype):
    z, ids, lq = make(N, V, K, seed=N + V + K, dtype=dtype)
    check(z, ids, lq, rest=rest)


@pytest.mark.gpu
@pytest.mark.parametrize("alpha", [(1.0, 0.0), (0.0, 1.0), (0.1, 0.9), (-0.5, 2.0), (0.0, 0.0)])
@pytest.mark.parametrize("T", [0.25, 1.0, 3.0])
def test_parts_and_temperatures(alpha, T):
    z, ids, lq = make(5, 3001, 17, seed=7)
    w = torch.tensor([1.0, 0.25, 0.0, -2.0, 3.0])
    check(z, ids, lq, T=T, alpha=alpha, weight=w)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,off", [(1, 0), (8, 0), (27, 3), (5, 7)])
def test_strides_and_offsets(pad, off, dtype):
    N, V = 4, 20011
    z, ids, lq = make(N, V, 30, seed=pad, dtype=dtype)
    buf = torch.full((N * (V + pad) + off,), float("nan"), dtype=dtype, device="cuda")
    zc = buf[off:].view(N, V + pad)[:, :V]
    zc.copy_(z)
    o = check(z, ids, lq, alpha=(0.5, 0.5), zc=zc)
    # into rows of other strides, and in place: the same bits, and nothing between the rows
    ob = torch.full((N * (V + 3) + 1,), 7.0, dtype=dtype, device="cuda")
    oc = ob[1:].view(N, V + 3)[:, :V]
    out = ds.DistillOutput(o.loss.clone(), o.parts.clone(), o.norm.clone(), oc)
    kw = dict(alpha=(0.5, 0.5))
    ds.distill_loss(zc, ids.cuda(), lq.cuda(), out=out, **kw)
    assert torch.equal(oc, o.grad_logits) and (ob[1:].view(N, V + 3)[:, V:] == 7.0).all() and ob[0] == 7.0
    want = ds.distill_grad(zc, ids.cuda(), lq.cuda(), o.norm, torch.ones(N, device="cuda"), **kw)
    again = zc.clone()
    assert torch.equal(ds.distill_grad(again, ids.cuda(), lq.cuda(), o.norm, torch.ones(N, device="cuda"), out=again,
                                       **kw), want)
    out.grad_logits = zc
    ds.distill_loss(zc, ids.cuda(), lq.cuda(), out=out, **kw)
    assert torch.equal(zc, o.grad_logits) and torch.equal(out.loss, o.loss) and torch.equal(out.norm, o.norm)
    assert torch.isnan(buf[off:].view(N, V + pad)[:, V:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [2000, 40000])
def test_masked_entries(V, dtype):
    z, ids, lq = make(6, V, 12, seed=17, dtype=dtype)
    g = torch.Generator().manual_seed(2)
    off = torch.rand(6, V, generator=g) < 0.5
    off.scatter_(1, ids.clamp(min=0).long(), False)
    z[off] = -math.inf
    z[1][off[1]] = torch.finfo(dtype).min
    z[2] = -math.inf
    z[2].scatter_(0, ids[2].long(), torch.randn(12, generator=g).to(dtype))     # the rest is masked
    z[3, int(ids[3, 0])] = -math.inf                                            # a teacher's token is masked
    z[4] = -math.inf                                                            # nothing is left
    z[5] = torch.finfo(dtype).min                                               # a uniform row
    for rest in (True, False):
        o = check(z, ids, lq, rest=rest)
        check(z, ids, lq, rest=rest, alpha=(0.0, 1.0))
        assert o.loss[3] == math.inf and o.loss[4] == math.inf


@pytest.mark.gpu
def test_a_rest_far_below_keeps_its_digits():
    # the rest's probability is about e^-60: its logarithm and its gradient are as exact as any other
    V, K = 5000, 4
    z, ids, lq = make(3, V, K, seed=19, pad=False)
    z.scatter_add_(1, ids.long(), torch.full((3, K), 60.0))
    check(z, ids, lq, alpha=(0.7, 0.3))


@pytest.mark.gpu
def test_teachers_without_entries_and_of_whole_mass():
    z, ids, lq = make(4, 1000, 6, seed=23)
    ids[0] = -1
    lq[1] = torch.tensor([0.0] + [-math.inf] * 5)                    # one token has it all
    lq[2] = torch.log(torch.full((6,), 0.25))                        # more than one in sum: no rest
    lq[3] = -math.inf
    o = check(z, ids, lq)
    assert abs(float(o.loss[0])) < 1e-6 and (o.grad_logits[0].abs() < 1e-6).all()
    check(z, ids, lq, rest=False, alpha=(0.4, 0.6))


@pytest.mark.gpu
def test_nan_and_infinite_logits_stay_in_their_rows():
    z, ids, lq = make(6, 9000, 10, seed=29)
    want = ds.distill_loss(z.cuda(), ids.cuda(), lq.cuda())
    z[1, 5], z[2, 7], z[3, int(ids[3, 1])], z[4, int(ids[4, 2])] = math.nan, math.inf, math.nan, math.inf
    o = ds.distill_loss(z.cuda(), ids.cuda(), lq.cuda())
    g = ds.distill_grad(z.cuda(), ids.cuda(), lq.cuda(), o.norm, torch.ones(6, device="cuda"))
    for x, y in ((o.loss, want.loss), (o.parts, want.parts), (o.grad_logits, want.grad_logits)):
        assert torch.isnan(x[1:5]).all() and torch.equal(x[0], y[0]) and torch.equal(x[5], y[5])
    assert torch.isnan(g[1:5]).all() and torch.isfinite(g[0]).all() and torch.isfinite(g[5]).all()
    w = torch.tensor([1.0, 0.0, 0.0, 0.0, 0.0, 1.0], device="cuda")  # padding rows are not read
    o = ds.distill_loss(z.cuda(), ids.cuda(), lq.cuda(), weight=w)
    assert (o.loss[1:5] == 0).all() and (o.grad_logits[1:5] == 0).all() and (o.norm[1:5] == 0).all()
    assert torch.equal(o.grad_logits[5], want.grad_logits[5])


@pytest.mark.gpu
def test_bad_ids_are_their_rows_alone():
    N, V, K = 6, 3000, 40
    z, ids, lq = make(N, V, K, seed=31)
    want = ds.distill_loss(z.cuda(), ids.cuda(), lq.cuda())
    ids[1, 3], ids[2, 39], ids[3, 39], ids[4, 0] = V, -2, ids[3, 0], ids[4, 33]
    ws = ds.DistillWorkspace(N, V, K)
    o = ds.distill_loss(z.cuda(), ids.cuda(), lq.cuda(), workspace=ws)
    assert ws.status() == 1
    for x, y in ((o.loss, want.loss), (o.parts, want.parts), (o.norm, want.norm), (o.grad_logits, want.grad_logits)):
        assert torch.isnan(x[1:5]).all() and torch.equal(x[0], y[0]) and torch.equal(x[5], y[5])
    g = ds.distill_grad(z.cuda(), ids.cuda(), lq.cuda(), want.norm, torch.ones(N, device="cuda"), workspace=ws)
    assert ws.status() == 1 and torch.isnan(g[1:5]).all() and torch.isfinite(g[0]).all()
    ids = ids.clone()
    good = ds.distill_loss(z.cuda()[5:], ids.cuda()[5:], lq.cuda()[5:], workspace=ws)
    assert ws.status() == 0 and torch.equal(good.loss, want.loss[5:])


@pytest.mark.gpu
def test_gradient_is_the_slope():
    # of the sum of the losses along random directions, by central differences in fp64 of the reference
    z, ids, lq = make(3, 700, 9, seed=37)
    g = torch.Generator().manual_seed(5)
    for alpha, rest in (((1.0, 0.0), True), ((0.3, 0.7), True), ((1.0, 0.0), False)):
        grad = ds.distill_loss(z.cuda(), ids.cuda(), lq.cuda(), alpha=alpha, rest=rest).grad_logits.double().cpu()
        for _ in range(3):
            v = torch.randn(3, 700, generator=g).double()
            h = 1e-5
            up, dn = (reference(z.double() + s * h * v, ids, lq, 1.0, alpha, rest, torch.ones(3))["loss"].sum()
                      for s in (1, -1))
            # differences are off by h^2 and by rounding over h (1e-10 either way), the gradient by its tolerance
            assert abs(float((up - dn) / (2 * h) - (grad * v).sum())) < 3e-5


@pytest.mark.gpu
def test_rows_have_the_same_bits_in_any_call():
    N, V, K = 300, 5000, 20
    z, ids, lq = make(N, V, K, seed=41)
    zc, ic, lc = z.cuda(), ids.cuda(), lq.cuda()
    big = ds.distill_loss(zc, ic, lc)
    for i in (0, 1, 150, 299):
        one = ds.distill_loss(zc[i:i + 1], ic[i:i + 1], lc[i:i + 1])
        assert torch.equal(one.loss, big.loss[i:i + 1]) and torch.equal(one.grad_logits, big.grad_logits[i:i + 1])
        assert torch.equal(one.norm, big.norm[i:i + 1])


@pytest.mark.gpu
def test_leading_shape_no_rows_and_a_shared_workspace():
    z, ids, lq = make(12, 3000, 8, seed=43)
    ws = ds.DistillWorkspace(64, 20000, 64)
    flat = ds.distill_loss(z.cuda(), ids.cuda(), lq.cuda(), workspace=ws)
    z2, i2, l2 = make(20, 20000, 64, seed=44)
    ds.distill_loss(z2.cuda(), i2.cuda(), l2.cuda(), workspace=ws)
    o = ds.distill_loss(z.cuda().view(3, 4, -1), ids.cuda().view(3, 4, -1), lq.cuda().view(3, 4, -1), workspace=ws)
    assert o.loss.shape == (3, 4) and o.norm.shape == (3, 4, 4) and o.grad_logits.shape == (3, 4, 3000)
    assert torch.equal(o.loss.view(-1), flat.loss) and torch.equal(o.grad_logits.view(12, -1), flat.grad_logits)
    none = ds.distill_loss(z.cuda()[:0], ids.cuda()[:0], lq.cuda()[:0])
    assert none.loss.shape == (0,) and none.grad_logits.shape == (0, 3000)


@pytest.mark.gpu
def test_captured_graphs_that_share_a_workspace():
    N, V, K = 9, 12000, 16
    ws = ds.DistillWorkspace(N, V, K)
    s = torch.cuda.Stream()
    plans, graphs = [], []
    for seed in (51, 52):
        z, ids, lq = (t.cuda() for t in make(N, V, K, seed=seed))
        torch.cuda.synchronize()
        plans.append((ds.DistillPlan(z, ids, lq, workspace=ws, stream=s), (z, ids, lq)))
    for plan, _ in plans:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            plan.run(s)
        graphs.append(g)
    for z, _, _ in (p[1] for p in plans):
        z.mul_(1.25)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for plan, (z, ids, lq) in plans:
        want = ds.distill_loss(z, ids, lq)
        assert torch.equal(plan.out.loss, want.loss) and torch.equal(plan.out.grad_logits, want.grad_logits)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    V, N = 1 << 24, 130                                              # N V > 2^31 entries
    z = torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
    z[N - 1, V - 1] = 20.0
    ids = torch.full((N, 1), V - 1, dtype=torch.int32, device="cuda")
    lq = torch.full((N, 1), math.log(0.5), device="cuda")
    o = ds.distill_loss(z, ids, lq)
    p = 1.0 / (1.0 + (V - 1) * math.exp(-20.0))
    want = 0.5 * (math.log(0.5) - math.log(p)) + 0.5 * (math.log(0.5) - math.log(1 - p))
    assert abs(float(o.loss[N - 1]) - want) < 1e-5
    assert abs(float(o.grad_logits[N - 1, V - 1]) - (p - 0.5)) < 2e-3
    assert abs(float(o.grad_logits[N - 1, 0]) / ((0.5 - p) / (V - 1)) - 1) < 6e-3


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_that_no_cluster_holds(dtype):
    # 4 and 3.5 MB: the loss and its gradient in three passes, the same bits in calls of one row
    V = (1 << 20) + 5 if dtype == torch.float32 else 1_800_003
    z, ids, lq = make(2, V, 100, seed=61, dtype=dtype)
    o = check(z, ids, lq, alpha=(0.3, 0.7), T=0.8)
    one = ds.distill_loss(z.cuda()[1:], ids.cuda()[1:], lq.cuda()[1:], alpha=(0.3, 0.7), T=0.8)
    assert torch.equal(one.loss, o.loss[1:]) and torch.equal(one.grad_logits, o.grad_logits[1:])


@pytest.mark.gpu
def test_loss_is_the_same_with_and_without_its_gradient():
    for V, dtype in ((30000, torch.float32), (151936, torch.bfloat16), (20003, torch.bfloat16)):
        z, ids, lq = make(5, V, 33, seed=V, dtype=dtype)
        a = ds.distill_loss(z.cuda(), ids.cuda(), lq.cuda(), alpha=(0.5, 0.5))
        b = ds.distill_loss(z.cuda(), ids.cuda(), lq.cuda(), alpha=(0.5, 0.5), want_grad=False)
        assert torch.equal(a.loss, b.loss) and torch.equal(a.parts, b.parts) and torch.equal(a.norm, b.norm)


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported(monkeypatch):
    z, ids, lq = make(3, 50000, 9, seed=67)
    ws = ds.DistillWorkspace(3, 50000, 9)
    want = ds.distill_loss(z.cuda(), ids.cuda(), lq.cuda(), workspace=ws)
    monkeypatch.setenv("DSPARK_TEST_STUCK_WAIT", "mbar")
    o = ds.distill_loss(z.cuda(), ids.cuda(), lq.cuda(), workspace=ws)
    assert ws.status() == 4 and torch.isnan(o.loss).all() and torch.isnan(o.grad_logits).all()
    monkeypatch.delenv("DSPARK_TEST_STUCK_WAIT")
    o = ds.distill_loss(z.cuda(), ids.cuda(), lq.cuda(), workspace=ws)
    assert ws.status() == 0 and torch.equal(o.loss, want.loss) and torch.equal(o.grad_logits, want.grad_logits)


@pytest.mark.gpu
def test_a_first_call_can_be_captured():
    # a length of row that no call has had: its shape is asked for under capture
    z, ids, lq = (t.cuda() for t in make(4, 27_777, 11, seed=71))
    s = torch.cuda.Stream()
    plan = ds.DistillPlan(z, ids, lq, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        plan.run(s)
    graph.replay()
    torch.cuda.synchronize()
    want = ds.distill_loss(z, ids, lq)
    assert torch.equal(plan.out.grad_logits, want.grad_logits) and torch.equal(plan.out.loss, want.loss)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5, 1031, 9001])
def test_the_gradient_alone_into_rows_of_any_alignment(V, dtype):
    z, ids, lq = make(3, V, 4, seed=61)
    z, ids, lq = z.to(dtype).cuda(), ids.cuda(), lq.cuda()
    o = ds.distill_loss(z, ids, lq)
    one = torch.ones(3, device="cuda")
    want = ds.distill_grad(z, ids, lq, o.norm, one)   # (rows aligned as the logits' are)
    for pad in range(8):
        for off in range(0, 8, 3):
            buf = torch.full((3 * (V + pad) + 16,), 7.0, dtype=dtype, device="cuda")
            out = buf[off:off + 3 * (V + pad)].view(3, V + pad)[:, :V]
            ds.distill_grad(z, ids, lq, o.norm, one, out=out)
            assert torch.equal(out, want), (pad, off)
            assert (buf[:off] == 7.0).all() and (buf[off + 3 * (V + pad) - pad:] == 7.0).all()
