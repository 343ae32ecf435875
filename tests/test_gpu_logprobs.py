"""Token log probabilities and their gradient against plain 64-bit forms.

Tolerances, from the arithmetic: with d = (z - max) / T, an exponential in fp32 is off by about
2^-22 + |d| 2^-23 of itself, so ln S is off by at most 2^-21 (1 + E|d|) and logp by that plus the
rounding of d: 2^-21 (4 + |d_x| + E|d|).  The entropy's two terms are off by 2^-21 (1 + E|d|^2) at
most.  The gradient's factor p is off by 2^-21 (4 + |ln p|) of itself, and bf16 results by 2^-8."""
import math

import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

EPS = 2.0 ** -21


def reference(z, tok, T, top):
    """Row by row in float64: logp, norm, entropy, rank, alternatives, and E|d|, E|d|^2."""
    z, N = z.double(), z.shape[0]
    r = dict(logp=torch.zeros(N), entropy=torch.zeros(N), m=torch.zeros(N), ls=torch.zeros(N),
             d1=torch.zeros(N), d2=torch.zeros(N), dx=torch.zeros(N))
    r = {k: v.double() for k, v in r.items()}
    rank = torch.zeros(N, dtype=torch.int32)
    ids = torch.full((N, top), -1, dtype=torch.int32)
    tlp = torch.full((N, top), -math.inf, dtype=torch.float64)
    for i in range(N):
        row, x = z[i], int(tok[i])
        some = row > -math.inf
        m = row.max() if some.any() else torch.tensor(-math.inf, dtype=torch.float64)
        d = torch.where(some, (row - m) / T, torch.tensor(-math.inf, dtype=torch.float64))
        e = torch.where(some, torch.exp(d), torch.zeros_like(d))
        S = e.sum()
        ls = torch.log(S) if some.any() else torch.tensor(0.0)
        p = e / S if some.any() else e
        fd = torch.where(p > 0, d, torch.zeros_like(d))
        r["m"][i], r["ls"][i] = m, ls
        r["entropy"][i] = (ls - (p * fd).sum()) if some.any() else 0.0
        r["d1"][i], r["d2"][i] = (p * fd.abs()).sum(), (p * fd * fd).sum()
        if x >= 0:
            rank[i] = int((row > row[x]).sum()) + 1
        # what fp32 cannot hold is -inf: the lowest number over a temperature below one
        d = torch.where(d < -torch.finfo(torch.float32).max, torch.full_like(d, -math.inf), d)
        if x >= 0:
            r["logp"][i] = d[x] - ls
            r["dx"][i] = d[x].abs()
        order = torch.sort(row + 0.0, descending=True, stable=True).indices
        order = order[row[order] > -math.inf][:top]
        ids[i, :len(order)] = order.to(torch.int32)
        tlp[i, :len(order)] = d[order] - ls
    return r, rank, ids, tlp


def close(name, got, want, tol):
    got, want = got.double().cpu(), want.double()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), name
    err = (got - want)[~inf].abs()
    tol = tol.expand_as(want)[~inf] if isinstance(tol, torch.Tensor) else tol
    assert (err <= tol).all(), (name, float((err - tol).max()), float(err.max()))


def check(z, tok, T=1.0, top=0, zc=None):
    """z: host logits [N, V] (the values the device sees), zc: the device tensor (default z on it)."""
    zc = z.cuda() if zc is None else zc
    N, V = z.shape
    ws = ds.LogprobWorkspace(N, V, top)
    for _ in range(2):  # the second call meets the workspace as the first one left it
        o = ds.token_logprobs(zc, tok.cuda(), T=T, top=top, workspace=ws)
    torch.cuda.synchronize()
    assert ws.status() == 0
    r, rank, ids, tlp = reference(z.float(), tok, T, top)
    tol = EPS * (4 + r["dx"] + r["d1"])
    close("logp", o.logp, r["logp"], torch.where(torch.isfinite(tol), tol, torch.ones_like(tol)))
    close("max", o.norm[..., 0], r["m"], 0.0)
    close("ln sum", o.norm[..., 1], r["ls"], EPS * (1 + r["d1"]))
    close("entropy", o.entropy, r["entropy"], EPS * (2 + 2 * r["d1"] + r["d2"]))
    assert torch.equal(o.rank.cpu(), rank)
    if top:
        assert torch.equal(o.top_ids.cpu(), ids)
        dk = torch.where(torch.isfinite(tlp), tlp.abs(), torch.zeros_like(tlp))
        close("top_logp", o.top_logp, tlp, EPS * (4 + 2 * dk + r["d1"][:, None]))
    return o


def make(N, V, dtype, seed, std=3.0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(N, V, generator=g) * std).to(dtype)
    tok = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    return z, tok


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,top", [(1, 2, 2), (1, 3, 1), (2, 31, 31), (3, 32, 32), (5, 1001, 7), (4, 4096, 32),
                                     (3, 8191, 20), (2, 8193, 20), (7, 16384, 5), (1, 50021, 32),
                                     (1, 151936, 5), (3, 151936, 0), (300, 1000, 3), (160, 33000, 6)])
def test_logprobs(N, V, top, dtype):
    z, tok = make(N, V, dtype, seed=N * 7 + V + top)
    check(z, tok, top=top)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0.25, 0.7, 1.5, 40.0])
def test_logprobs_temperature(T):
    z, tok = make(4, 9999, torch.float32, seed=11)
    check(z, tok, T=T, top=10)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,off", [(1, 0), (8, 0), (27, 3), (5, 7)])
def test_logprobs_row_strides_and_offsets(pad, off, dtype):
    # rows of a padded vocabulary, starting at any element; the padding holds what must not be read
    N, V = 6, 20011
    z, tok = make(N, V, dtype, seed=21 + pad)
    buf = torch.full((N * (V + pad) + off,), float("nan"), dtype=dtype, device="cuda")
    zc = buf[off:].view(N, V + pad)[:, :V]
    zc.copy_(z)
    check(z, tok, top=9, zc=zc)


@pytest.mark.gpu
def test_logprobs_leading_shape():
    z, tok = make(12, 3000, torch.float32, seed=31)
    flat = check(z, tok, top=4)
    o = ds.token_logprobs(z.cuda().view(3, 4, 3000), tok.cuda().view(3, 4), top=4)
    assert o.logp.shape == (3, 4) and o.norm.shape == (3, 4, 2) and o.top_ids.shape == (3, 4, 4)
    for a, b in [(o.logp, flat.logp), (o.norm, flat.norm), (o.top_ids, flat.top_ids), (o.rank, flat.rank)]:
        assert torch.equal(a.reshape(b.shape), b)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logprobs_ties_go_to_the_lower_entry(dtype):
    V = 30000
    g = torch.Generator().manual_seed(41)
    z = torch.stack([torch.zeros(V), torch.randint(0, 3, (V,), generator=g).float(),
                     torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0), torch.full((V,), -7.5)]).to(dtype)
    check(z, torch.tensor([0, 17, V - 1, 12345], dtype=torch.int32), top=32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logprobs_sorted_rows(dtype):
    # ascending, descending and clustered rows: the alternatives all sit side by side
    V = 40000
    up = torch.linspace(-20.0, 20.0, V)
    one = torch.randn(V, generator=torch.Generator().manual_seed(43))
    one[1024:2048] += 100.0
    z = torch.stack([up, up.flip(0), one]).to(dtype)
    check(z, torch.tensor([V - 1, 5, 1500], dtype=torch.int32), top=32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [0.5, 1.0])
def test_logprobs_masks(dtype, T):
    V, low = 20000, torch.finfo(dtype).min
    z, tok = make(8, V, dtype, seed=51)
    z[0] = -math.inf                               # nothing is left
    z[1] = low                                     # every entry is the lowest number: uniform
    z[2] = -math.inf
    z[2, 777] = -3.0                               # one entry left
    z[3] = -math.inf
    z[3, 19999] = low                              # one entry left, the lowest number
    z[4, ::2] = -math.inf                          # the given token is masked
    z[5, 1::2] = low
    z[6] = low
    z[6, 5:9] = 1.0
    z[7, 4:] = -math.inf                           # fewer entries than alternatives
    tok[2], tok[3], tok[4], tok[6], tok[7] = 777, 19999, 10, 6, 2
    o = check(z, tok, T=T, top=8)
    assert float(o.logp[0]) == -math.inf and float(o.entropy[0]) == 0.0 and int(o.rank[0]) == 1
    assert int(o.top_ids[0, 0]) == -1 and int(o.top_ids[7, 4]) == -1
    assert abs(float(o.logp[1]) + math.log(V)) < 1e-4


@pytest.mark.gpu
def test_logprobs_no_token_and_invalid_token():
    z, tok = make(6, 5000, torch.float32, seed=61)
    good = ds.token_logprobs(z.cuda(), tok.cuda(), top=3)
    bad = tok.clone()
    bad[1], bad[2], bad[4] = -1, 5000, -7
    ws = ds.LogprobWorkspace(6, 5000, 3)
    o = ds.token_logprobs(z.cuda(), bad.cuda(), top=3, workspace=ws)
    assert ws.status() == 1 and ws.status() == 0
    assert float(o.logp[1]) == 0.0 and int(o.rank[1]) == 0
    assert torch.isnan(o.logp[[2, 4]]).all() and o.rank[[2, 4]].tolist() == [-1, -1]
    for i in (0, 3, 5):
        assert o.logp[i] == good.logp[i] and o.rank[i] == good.rank[i]
    assert torch.equal(o.entropy, good.entropy) and torch.equal(o.top_ids, good.top_ids)


@pytest.mark.gpu
def test_logprobs_nan_and_inf_rows():
    z, tok = make(5, 9000, torch.float32, seed=71)
    z[1, 4321] = math.nan
    z[2, 8999] = math.inf
    z[3] = math.nan
    good = ds.token_logprobs(make(5, 9000, torch.float32, seed=71)[0].cuda(), tok.cuda(), top=4)
    ws = ds.LogprobWorkspace(5, 9000, 4)
    o = ds.token_logprobs(z.cuda(), tok.cuda(), top=4, workspace=ws)
    assert ws.status() == 0
    assert torch.isnan(o.logp[[1, 2, 3]]).all() and torch.isnan(o.entropy[[1, 2, 3]]).all()
    assert 4321 not in o.top_ids[1].tolist() and int(o.top_ids[2, 0]) == 8999
    assert o.top_ids[3].tolist() == [-1] * 4
    for i in (0, 4):
        assert o.logp[i] == good.logp[i] and torch.equal(o.top_ids[i], good.top_ids[i])


@pytest.mark.gpu
def test_logprobs_repeat_identical_and_other_stream():
    z, tok = make(9, 60000, torch.bfloat16, seed=81)
    zc, tc = z.cuda(), tok.cuda()
    a = ds.token_logprobs(zc, tc, top=6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = ds.token_logprobs(zc, tc, top=6, stream=s)
    s.synchronize()
    for x, y in [(a.logp, b.logp), (a.norm, b.norm), (a.entropy, b.entropy), (a.rank, b.rank),
                 (a.top_ids, b.top_ids), (a.top_logp, b.top_logp)]:
        assert torch.equal(x, y)


@pytest.mark.gpu
def test_logprobs_in_a_graph():
    z, tok = make(8, 151936, torch.bfloat16, seed=83)
    plan = ds.LogprobPlan(z.cuda(), tok.cuda(), top=5)
    plan.run()
    torch.cuda.synchronize()
    want = plan.out.logp.clone(), plan.out.top_ids.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run(torch.cuda.current_stream())
    for _ in range(3):
        plan.out.logp.zero_()
        plan.out.top_ids.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(plan.out.logp, want[0]) and torch.equal(plan.out.top_ids, want[1])


@pytest.mark.gpu
def test_logprobs_no_rows():
    z = torch.empty(0, 100, device="cuda")
    o = ds.token_logprobs(z, torch.empty(0, dtype=torch.int32, device="cuda"), top=2)
    assert o.logp.shape == (0,) and o.top_ids.shape == (0, 2)


@pytest.mark.gpu
def test_logprobs_rows_past_32_bit_offsets():
    # the last rows start more than 2^32 elements into the logits
    N, V = 17000, 262144
    z = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")
    z[:2].normal_()
    z[-2:].normal_()
    z[2:-2] = z[0]
    tok = torch.full((N,), V - 1, dtype=torch.int32, device="cuda")
    o = ds.token_logprobs(z, tok, top=1)
    few = ds.token_logprobs(z[-2:].clone(), tok[-2:], top=1)
    assert torch.equal(o.logp[-2:], few.logp) and torch.equal(o.top_ids[-2:], few.top_ids)
    assert torch.equal(o.logp[2:-2], o.logp[:1].expand(N - 4))


# ------------------------------------------------------------------ gradient
def formula(z, tok, T, gl, gh):
    """dL/dz in float64, and the scale and ln p that the tolerance uses."""
    z = z.double()
    some = z > -math.inf
    m = torch.where(some.any(1), z.amax(1), torch.zeros(z.shape[0], dtype=torch.float64))[:, None]
    d = (z - m) / T
    e = torch.where(some, torch.exp(d), torch.zeros_like(d))
    S = e.sum(1, keepdim=True)
    p = torch.where(S > 0, e / S.clamp(min=1e-300), torch.zeros_like(e))
    lp = torch.where(p > 0, d - torch.log(S.clamp(min=1e-300)), torch.zeros_like(d))
    H = -(p * lp).sum(1, keepdim=True)
    hot = torch.zeros_like(z)
    on = (tok >= 0).nonzero()[:, 0]
    hot[on, tok[on].long()] = 1.0
    g = torch.where(tok >= 0, gl.double(), torch.zeros(len(tok), dtype=torch.float64))[:, None]
    h = gh.double()[:, None]
    grad = (g * (hot - p) - h * p * (lp + H)) / T
    size = (g.abs() * (hot + p) + h.abs() * p * (lp.abs() + H + 1)) / T
    return grad, size, lp


def check_grad(z, tok, T, gl, gh, zc=None, out=None):
    zc = z.cuda() if zc is None else zc
    o = ds.token_logprobs(zc, tok.cuda(), T=T)
    got = ds.token_logprobs_grad(zc, tok.cuda(), o.norm, T=T, grad_logp=None if gl is None else gl.cuda(),
                                 grad_entropy=None if gh is None else gh.cuda(),
                                 entropy=o.entropy, out=out)
    N = z.shape[0]
    want, size, lp = formula(z.float(), tok, T, gl if gl is not None else torch.zeros(N),
                             gh if gh is not None else torch.zeros(N))
    tol = size * (2 * EPS * (6 + lp.abs() + 1 / T) + (2.0 ** -8 if z.dtype == torch.bfloat16 else 0)) + 1e-36
    close("grad", got, want, tol)
    return got


def test_gradient_formula_against_differences():
    """The 64-bit formula itself, by central differences of the 64-bit forward pass."""
    g = torch.Generator().manual_seed(5)
    z = torch.randn(3, 9, generator=g, dtype=torch.float64)
    z[1, 4] = -math.inf
    tok = torch.tensor([2, 0, -1], dtype=torch.int32)
    gl, gh = torch.randn(3, generator=g).double(), torch.randn(3, generator=g).double()
    T = 0.8

    def loss(q):
        r = reference(q, tok, T, 0)[0]
        return (torch.where(tok >= 0, gl, torch.zeros_like(gl)) * r["logp"] + gh * r["entropy"]).sum()

    want, _, _ = formula(z, tok, T, gl, gh)
    for i in range(3):
        for v in range(9):
            if z[i, v] == -math.inf:
                assert want[i, v] == 0
                continue
            q = z.clone()
            q[i, v] += 1e-5
            up = loss(q)
            q[i, v] -= 2e-5
            assert abs((up - loss(q)) / 2e-5 - want[i, v]) < 1e-8


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,T", [(1, 2, 1.0), (3, 33, 0.7), (5, 1001, 1.0), (4, 8192, 1.3), (2, 8200, 1.0),
                                   (3, 50021, 0.6), (2, 151936, 1.0)])
def test_gradient(N, V, T, dtype):
    z, tok = make(N, V, dtype, seed=91 + V)
    g = torch.Generator().manual_seed(V)
    check_grad(z, tok, T, torch.randn(N, generator=g), torch.randn(N, generator=g))
    check_grad(z, tok, T, torch.randn(N, generator=g), None)
    check_grad(z, tok, T, None, torch.randn(N, generator=g))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_masks_and_missing_tokens(dtype):
    V = 7000
    z, tok = make(7, V, dtype, seed=95)
    z[0] = -math.inf
    z[1] = torch.finfo(dtype).min
    z[2, 10:] = -math.inf
    z[3, ::2] = torch.finfo(dtype).min
    z[4, 5:] = -math.inf
    z[4, :5] = torch.finfo(dtype).min
    tok[2], tok[4], tok[5] = 3, 2, -1
    g = torch.Generator().manual_seed(96)
    check_grad(z, tok, 0.5, torch.randn(7, generator=g), torch.randn(7, generator=g))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,gpad,off", [(5, 0, 0), (0, 3, 1), (8, 8, 0), (3, 3, 2), (16, 8, 5)])
def test_gradient_strides(pad, gpad, off, dtype):
    N, V = 5, 6001
    z, tok = make(N, V, dtype, seed=97)
    buf = torch.full((N * (V + pad) + off,), float("nan"), dtype=dtype, device="cuda")
    zc = buf[off:].view(N, V + pad)[:, :V]
    zc.copy_(z)
    obuf = torch.full((N, V + gpad), 7.0, dtype=dtype, device="cuda")
    g = torch.Generator().manual_seed(98)
    check_grad(z, tok, 1.0, torch.randn(N, generator=g), torch.randn(N, generator=g), zc=zc, out=obuf[:, :V])
    assert (obuf[:, V:] == 7.0).all()          # the output's padding is not touched


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_in_place(dtype):
    z, tok = make(3, 12345, dtype, seed=99)
    gl = torch.randn(3, generator=torch.Generator().manual_seed(1))
    apart = check_grad(z, tok, 1.0, gl, None)
    zc = z.cuda()
    o = ds.token_logprobs(zc, tok.cuda())
    ds.token_logprobs_grad(zc, tok.cuda(), o.norm, grad_logp=gl.cuda(), out=zc)
    assert torch.equal(zc, apart)


@pytest.mark.gpu
def test_gradient_invalid_token():
    z, tok = make(3, 400, torch.float32, seed=100)
    o = ds.token_logprobs(z.cuda(), tok.cuda())
    tok[1] = 400
    got = ds.token_logprobs_grad(z.cuda(), tok.cuda(), o.norm, grad_logp=torch.ones(3, device="cuda"))
    assert torch.isnan(got[1]).all() and not torch.isnan(got[[0, 2]]).any()


@pytest.mark.gpu
def test_refusals():
    z, tok = make(4, 100, torch.float32, seed=101)
    z, tok = z.cuda(), tok.cuda()
    norm = torch.zeros(4, 2, device="cuda")
    one = torch.ones(4, device="cuda")
    with pytest.raises(ValueError):
        ds.token_logprobs(z.cpu(), tok)
    with pytest.raises(TypeError):
        ds.token_logprobs(z.half(), tok)
    with pytest.raises(TypeError):
        ds.token_logprobs(z, tok.long())
    with pytest.raises(ValueError):
        ds.token_logprobs(z, tok[:3])
    with pytest.raises(ValueError):
        ds.token_logprobs(z.t().contiguous().t(), tok)
    with pytest.raises(ValueError):
        ds.token_logprobs(z[:1].expand(4, 100), tok)
    with pytest.raises(ValueError):
        ds.token_logprobs(z, tok, top=33)
    with pytest.raises(ds._lib.DsparkError):
        ds.token_logprobs(z, tok, T=0.0)
    with pytest.raises(ds._lib.DsparkError):     # a workspace of a smaller problem
        small = ds.LogprobWorkspace(4, 100, 0)
        small.nbytes = 128
        ds.token_logprobs(z, tok, top=5, workspace=small)
    with pytest.raises(ValueError):
        ds.token_logprobs_grad(z, tok, norm)
    with pytest.raises(ValueError):
        ds.token_logprobs_grad(z, tok, norm, grad_entropy=one)
    with pytest.raises(ValueError):
        ds.token_logprobs_grad(z, tok, norm[:2], grad_logp=one)
    with pytest.raises(ValueError):
        ds.token_logprobs_grad(z, tok, norm, grad_logp=torch.ones(1, device="cuda").expand(4))
