"""Penalties, biases and masks on logits, and their gradient, against plain 64-bit forms.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32): the quotient or product by the
repetition penalty is off by u of itself, the two subtractions and each addition of a bias by u of
their results, all of which are at most A = |z scale| + f c + p + sum |bias|; so an entry is off by
at most u (4 + its biases) A, and a bf16 result by 2^-8 of itself beside.  Entries that nothing
touches keep their bits."""
import math

import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

U = 2.0 ** -24
NAMES = ("history", "lengths", "prompt_lengths", "drafted", "repetition", "presence", "frequency", "bias_tokens",
         "bias", "mask", "mask_rows")


def pack(allowed, words=None):
    """Bits [M, V] to words [M, >= ceil(V / 32)] int32."""
    M, V = allowed.shape
    W = words or (V + 31) // 32
    bits = torch.zeros(M, W * 32, dtype=torch.int64)
    bits[:, :V] = allowed
    w = (bits.view(M, W, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def allowed_rows(x, N, V):
    ok = torch.ones(N, V, dtype=torch.bool)
    if x.get("mask") is None:
        return ok
    rows = x["mask_rows"].reshape(-1) if x.get("mask_rows") is not None else torch.arange(N)
    for i in range(N):
        if rows[i] >= 0:
            m = x["mask"][int(rows[i])].long() & 0xFFFFFFFF
            v = torch.arange(V)
            ok[i] = (m[v // 32] >> (v % 32)) & 1 == 1
    return ok


def reference(z, x, grad=None):
    """(values, bound on the error, touched) of every entry in float64, request by request."""
    three = z.dim() == 3
    zz = z.double() if three else z.double()[:, None]
    B, R, V = zz.shape
    y, A, touched = zz.clone(), torch.zeros(B, R, V, dtype=torch.float64), torch.zeros(B, R, V, dtype=torch.bool)
    g = None if grad is None else (grad.double() if three else grad.double()[:, None]).clone()
    for b in range(B):
        get = lambda n, d: float(x[n][b]) if x.get(n) is not None else d
        rho, pres, freq = get("repetition", 1.0), get("presence", 0.0), get("frequency", 0.0)
        h = x["history"][b].tolist() if x.get("history") is not None else []
        h = h[:int(x["lengths"][b])] if x.get("lengths") is not None else h
        P = int(x["prompt_lengths"][b]) if x.get("prompt_lengths") is not None else 0
        seen = {t for t in h if t >= 0}
        count = {}
        for t in h[P:]:
            count[t] = count.get(t, 0) + 1
        add, mag, dup = {}, {}, {}
        if x.get("bias") is not None:
            for t, v in zip(x["bias_tokens"][b].tolist(), x["bias"][b].tolist()):
                if t >= 0:
                    add[t] = add.get(t, 0.0) + v
                    mag[t] = mag.get(t, 0.0) + abs(v)
                    dup[t] = dup.get(t, 0) + 1
        for r in range(R):
            if r and x.get("drafted") is not None and int(x["drafted"][b, r - 1]) >= 0:
                t = int(x["drafted"][b, r - 1])
                seen.add(t)
                count[t] = count.get(t, 0) + 1
            for t in seen | set(add):
                v = zz[b, r, t]
                s = (1.0 / rho if v > 0 else rho) if t in seen else 1.0
                c = count.get(t, 0)
                y[b, r, t] = v * s - freq * c - (pres if c > 0 else 0.0) + add.get(t, 0.0)
                # (an infinite logit or bias decides its entry: no bound)
                size = float(v.abs()) * s + abs(freq) * c + abs(pres) + mag.get(t, 0.0)
                A[b, r, t] = U * (4 + dup.get(t, 0)) * size if math.isfinite(size) else 0.0
                touched[b, r, t] = True
                if g is not None:
                    g[b, r, t] *= s
    ok = allowed_rows(x, B * R, V).view(B, R, V)
    if g is not None:
        g = torch.where(ok, g, torch.zeros_like(g))
        return g.view(z.shape), (U * g.abs()).view(z.shape), (touched & ok).view(z.shape), ok.view(z.shape)
    y = torch.where(ok, y, torch.full_like(y, -math.inf))
    return y.view(z.shape), A.view(z.shape), (touched & ok).view(z.shape), ok.view(z.shape)


def same(got, want, tol):
    """got within tol of want, the same infinities, NaN where want has NaN."""
    got, want = got.double().cpu(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])
    err = (got - want)[fine].abs()
    assert (err <= tol[fine]).all(), (float((err - tol[fine]).max()), float(err.max()))


def dev(x):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}


def check(z, x, dtype=None, zc=None, out=None):
    zc = z.cuda() if zc is None else zc
    want, A, touched, ok = reference(z.float(), x)
    odt = dtype or z.dtype
    got = ds.process_logits(zc, dtype=dtype if out is None else None, out=out, **dev(x))
    assert got.shape == z.shape and got.dtype == odt
    g = got.cpu()
    big = torch.finfo(odt).max
    want = torch.where(want.abs() > big * (1 + 2.0 ** -9), torch.sign(want) * math.inf, want)
    rnd = 2.0 ** -8 if odt == torch.bfloat16 else U
    tol = A + torch.where(torch.isfinite(want), want.abs(), torch.zeros_like(want)) * (0.0 if odt == z.dtype else rnd)
    if odt == torch.bfloat16:
        tol = A * 1.01 + torch.where(torch.isfinite(want), want.abs(), torch.zeros_like(want)) * 2.0 ** -8 * touched
        tol += (~touched) * (torch.where(torch.isfinite(want), want.abs(), torch.zeros_like(want))
                             * (2.0 ** -8 if z.dtype == torch.float32 else 0.0))
    same(g, want, tol)
    plain = ok & ~touched
    assert torch.equal(g[plain].view(torch.int16 if odt == torch.bfloat16 else torch.int32),
                       z.to(odt)[plain].view(torch.int16 if odt == torch.bfloat16 else torch.int32))
    return got


def make(B, R, V, H, seed, dtype=torch.float32, nb=0, masked=0, flat=False, std=3.0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(B, R, V, generator=g) * std).to(dtype)
    x = dict(history=torch.randint(0, min(V, max(4, H // 2 + 1)), (B, H), generator=g, dtype=torch.int32),
             lengths=torch.randint(0, H + 1, (B,), generator=g, dtype=torch.int32),
             repetition=1.0 + torch.rand(B, generator=g), presence=torch.rand(B, generator=g),
             frequency=torch.rand(B, generator=g))
    x["prompt_lengths"] = (torch.rand(B, generator=g) * (x["lengths"] + 1)).to(torch.int32).clamp(max=x["lengths"])
    x["drafted"] = torch.randint(-1, min(V, 12), (B, R - 1), generator=g, dtype=torch.int32)
    if nb:
        x["bias_tokens"] = torch.randint(-1, min(V, 2 * nb), (B, nb), generator=g, dtype=torch.int32)
        x["bias"] = 5.0 * torch.randn(B, nb, generator=g)
    if masked:
        x["mask"] = pack(torch.rand(masked, V, generator=g) < torch.linspace(0.01, 0.99, masked)[:, None])
        x["mask_rows"] = torch.randint(-1, masked, (B, R), generator=g, dtype=torch.int32)
    if flat:
        z, x["drafted"] = z[:, 0], x["drafted"][:, :0]
        if masked:
            x["mask_rows"] = x["mask_rows"][:, 0].contiguous()
    return z, x


TYPES = [(torch.float32, None), (torch.bfloat16, None), (torch.bfloat16, torch.float32),
         (torch.float32, torch.bfloat16)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("B,R,V,H,nb,masked", [(1, 1, 2, 3, 1, 1), (1, 1, 3, 0, 0, 2), (2, 3, 31, 5, 2, 2),
                                               (1, 2, 32, 40, 0, 1), (3, 8, 33, 1, 4, 3), (2, 5, 1001, 900, 40, 3),
                                               (5, 1, 4096, 64, 0, 0), (1, 4, 4097, 5000, 7, 2),
                                               (2, 2, 8191, 300, 300, 4), (1, 17, 12289, 77, 33, 5),
                                               (1, 1, 50021, 20000, 1, 1), (4, 32, 700, 50, 3, 9)])
def test_process(B, R, V, H, nb, masked, dtype, out):
    z, x = make(B, R, V, H, seed=B + 3 * R + V + H, dtype=dtype, nb=nb, masked=masked)
    check(z, x, dtype=out)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_single_tokens(dtype):
    z, x = make(9, 1, 6000, 200, seed=3, dtype=dtype, nb=10, masked=4, flat=True)
    check(z, x)


@pytest.mark.gpu
@pytest.mark.parametrize("keep", [(), ("repetition", "history"), ("presence", "history"), ("frequency", "drafted"),
                                  ("bias_tokens", "bias"), ("mask", "mask_rows"), ("history", "lengths"),
                                  ("repetition", "drafted", "history", "prompt_lengths", "lengths")])
def test_each_tool_alone(keep):
    z, x = make(3, 4, 5000, 60, seed=5, nb=9, masked=3)
    check(z, {k: v for k, v in x.items() if k in keep})


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("pad,off,opad,ooff", [(0, 0, 3, 1), (1, 0, 0, 0), (27, 3, 0, 2), (5, 7, 8, 5), (8, 0, 8, 0),
                                               (3, 6, 3, 6)])
def test_strides_and_offsets(pad, off, opad, ooff, dtype, out):
    # padded rows from any element on, read and written; what lies between the rows stays as it was
    B, R, V = 2, 3, 9001
    z, x = make(B, R, V, 500, seed=pad + off, dtype=dtype, nb=5, masked=2)
    odt = out or dtype
    zb = torch.full((B * R * (V + pad) + off,), float("nan"), dtype=dtype, device="cuda")
    zc = zb[off:].view(B, R, V + pad)[..., :V]
    zc.copy_(z)
    ob = torch.full((B * R * (V + opad) + ooff,), 7.0, dtype=odt, device="cuda")
    oc = ob[ooff:].view(B, R, V + opad)[..., :V]
    check(z, x, dtype=odt, zc=zc, out=oc)
    assert (ob[:ooff] == 7.0).all() and (ob[ooff:].view(B, R, V + opad)[..., V:] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off", [0, 3])
@pytest.mark.parametrize("drop", [(), ("mask", "mask_rows"),
                                  ("repetition", "presence", "frequency", "bias_tokens", "bias")])
def test_in_place(dtype, off, drop):
    B, R, V = 3, 2, 10007
    z, x = make(B, R, V, 300, seed=11, dtype=dtype, nb=6, masked=3)
    x = {k: v for k, v in x.items() if k not in drop}
    want = check(z, x)
    buf = torch.zeros(B * R * V + off, dtype=dtype, device="cuda")
    zc = buf[off:].view(B, R, V)
    zc.copy_(z)
    got = ds.process_logits(zc, out=zc, **dev(x))
    assert got.data_ptr() == zc.data_ptr() and torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_special_values(dtype):
    V = 5000
    z, x = make(2, 3, V, 100, seed=21, dtype=dtype, nb=4, masked=2)
    lo = torch.finfo(dtype).min
    z[:, :, 0], z[:, :, 1], z[:, :, 2], z[:, :, 3] = -math.inf, lo, 0.0, -0.0
    z[:, :, 4], z[:, :, 5] = math.inf, float("nan")
    z[0, 1] = -math.inf
    x["history"][:, :6] = torch.arange(6, dtype=torch.int32)
    x["lengths"][:] = 50
    x["prompt_lengths"][:] = 3
    x["bias_tokens"][:, 0], x["bias"][:, 0] = 77, -math.inf           # a banned token
    check(z, x)


@pytest.mark.gpu
def test_rows_that_nothing_is_left_of():
    z, x = make(2, 2, 3000, 20, seed=23)
    x["mask"] = torch.zeros(1, 94, dtype=torch.int32)
    x["mask_rows"] = torch.tensor([[0, -1], [-1, 0]], dtype=torch.int32)
    got = check(z, x).cpu()
    assert (got[0, 0] == -math.inf).all() and (got[1, 1] == -math.inf).all() and torch.isfinite(got[0, 1]).all()
    o = ds.token_logprobs(got.cuda(), torch.zeros(2, 2, dtype=torch.int32, device="cuda"))
    assert o.entropy[0, 0] == 0.0 and o.logp[0, 0] == -math.inf


@pytest.mark.gpu
def test_mask_without_rows_and_wider_words():
    z, x = make(2, 2, 1000, 20, seed=25)
    g = torch.Generator().manual_seed(1)
    x["mask"] = pack(torch.rand(4, 1000, generator=g) < 0.5, words=40)
    check(z, x)
    x["mask"] = x["mask"].cuda()[:, :32].cpu()
    mask = torch.zeros(4, 64, dtype=torch.int32, device="cuda")[:, :32]
    mask.copy_(x["mask"])                                              # rows further apart than their words
    want = ds.process_logits(z.cuda(), **dev(x))
    assert torch.equal(ds.process_logits(z.cuda(), **{**dev(x), "mask": mask}), want)


@pytest.mark.gpu
def test_counts_of_one_token_and_of_all():
    V = 4500
    z = torch.randn(3, 2, V)
    h = torch.stack([torch.full((9000,), 4321), torch.arange(9000) % V, torch.full((9000,), -1)]).to(torch.int32)
    x = dict(history=h, repetition=torch.tensor([1.5, 0.5, 2.0]), presence=torch.tensor([0.1, -0.2, 0.3]),
             frequency=torch.tensor([0.01, -0.02, 0.5]), drafted=torch.tensor([[4321], [7], [-1]], dtype=torch.int32))
    check(z, x)


@pytest.mark.gpu
def test_drafted_token_twice_and_biases_of_one_token():
    V = 2000
    z = torch.randn(1, 9, V)
    x = dict(drafted=torch.tensor([[5, 5, 1999, -1, 5, 0, 1999, 5]], dtype=torch.int32),
             repetition=torch.tensor([1.25]), presence=torch.tensor([0.5]), frequency=torch.tensor([0.25]),
             bias_tokens=torch.tensor([[5] * 40 + [0, 1999, 5, -1, 0] + [1999] * 33], dtype=torch.int32),
             bias=torch.randn(1, 78))
    a = check(z, x)
    b = check(z, x)
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_bad_tokens_lengths_and_masks_are_nan():
    V, B = 3000, 7
    z, x = make(B, 3, V, 30, seed=31, nb=3, masked=2)
    x["lengths"][:], x["prompt_lengths"][:] = 30, 2
    good = ds.process_logits(z.cuda(), **dev(x)).cpu()
    x["history"][0, 29] = V
    x["history"][1, 4] = -2
    x["drafted"][2, 1] = V + 5
    x["bias_tokens"][3, 2] = V
    x["lengths"][4] = 31
    x["prompt_lengths"][5] = 31
    x["mask_rows"][6, 1] = 2
    got = ds.process_logits(z.cuda(), **dev(x)).cpu()
    assert torch.isnan(got[:6]).all() and torch.isnan(got[6, 1]).all()
    assert torch.equal(got[6, 0], good[6, 0]) and torch.equal(got[6, 2], good[6, 2])
    # what lies behind a text's length is not read
    x = {k: v.clone() for k, v in x.items()}
    x["history"][0, 29], x["lengths"][0] = V, 29
    assert not torch.isnan(ds.process_logits(z.cuda(), **dev(x))[0]).any()


@pytest.mark.gpu
def test_history_of_a_larger_buffer_and_no_request():
    z, x = make(3, 2, 4000, 50, seed=33)
    want = ds.process_logits(z.cuda(), **dev(x))
    buf = torch.full((3, 4096), 10 ** 9, dtype=torch.int32, device="cuda")
    buf[:, :50] = x["history"].cuda()
    assert torch.equal(ds.process_logits(z.cuda(), **{**dev(x), "history": buf[:, :50]}), want)
    assert torch.equal(ds.process_logits(z.cuda(), **{**dev(x), "history": buf}), want)
    none = ds.process_logits(z.cuda()[:0], **{k: v[:0] for k, v in dev(x).items()})
    assert none.shape == (0, 2, 4000)


@pytest.mark.gpu
@pytest.mark.parametrize("gdt,dtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                       (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("B,R,V,H,masked", [(1, 1, 2, 1, 1), (2, 7, 999, 400, 3), (3, 2, 8200, 64, 0), (1, 3, 20011, 9000, 2)])
def test_gradient(B, R, V, H, masked, gdt, dtype):
    z, x = make(B, R, V, H, seed=41 + V, dtype=dtype, masked=masked)
    x = {k: v for k, v in x.items() if k not in ("presence", "frequency")}
    z[..., 0] = 0.0
    g = torch.randn(B, R, V, generator=torch.Generator().manual_seed(9)).to(gdt)
    want, tol, touched, ok = reference(z.float(), x, grad=g.float())
    got = ds.process_logits_grad(g.cuda(), z.cuda(), **dev(x))
    assert got.dtype == dtype
    rounds = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    same(got, want, tol * 1.01 + want.abs() * rounds)
    if gdt == dtype:
        gc = g.cuda()
        assert torch.equal(ds.process_logits_grad(gc, z.cuda(), out=gc, **dev(x)), got)


@pytest.mark.gpu
def test_gradient_is_the_slope():
    # the processed logits are linear between the kinks: differences over a step that crosses none are exact
    # but for the rounding of the two ends (2 u |y| / step each)
    z, x = make(2, 3, 2500, 300, seed=51, masked=2)
    z = torch.where(z.abs() < 0.1, torch.full_like(z, 0.5), z)
    step = 2.0 ** -6
    hi, lo = (ds.process_logits((z + s * step).cuda(), **dev(x)).double().cpu() for s in (1, -1))
    w = {k: v for k, v in x.items() if k not in ("presence", "frequency")}
    g = ds.process_logits_grad(torch.ones(z.shape, device="cuda"), z.cuda(), **dev(w)).double().cpu()
    fine = torch.isfinite(hi)
    assert (g[~fine] == 0).all()
    slope = ((hi - lo) / (2 * step))[fine]
    bound = U * (5 * (hi.abs() + 5)[fine]) / step + 3 * U
    assert ((slope - g[fine]).abs() <= bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("B,R,V,H,nb", [(1, 1, 5000, 30000, 0), (2, 1, 40001, 70000, 40), (1, 2, 3000, 60000, 5),
                                        (3, 4, 9000, 66000, 3)])
def test_long_texts(B, R, V, H, nb):
    # texts that are counted in 16 and in 32 bits, by blocks of both sizes
    z, x = make(B, R, V, H, seed=H, nb=nb, masked=2)
    x["lengths"][0] = H
    x["history"][0, :] = 17                                          # one token tens of thousands of times
    x["history"][0, ::3] = V - 1
    check(z, x)
    w = {k: v for k, v in x.items() if k not in ("presence", "frequency", "bias", "bias_tokens")}
    g = torch.randn(B, R, V, generator=torch.Generator().manual_seed(9))
    want, tol, _, _ = reference(z, w, grad=g)
    same(ds.process_logits_grad(g.cuda(), z.cuda(), **dev(w)), want, tol * 1.01)


@pytest.mark.gpu
def test_many_biases_of_one_slice_and_repeats_across_steps():
    V, nb = 3000, 1024
    g = torch.Generator().manual_seed(2)
    z = torch.randn(2, 2, V, generator=g)
    x = dict(bias_tokens=torch.randint(-1, 300, (2, nb), generator=g, dtype=torch.int32), bias=torch.randn(2, nb, generator=g),
             history=torch.randint(0, 600, (2, 50), generator=g, dtype=torch.int32), frequency=torch.tensor([0.5, 0.0]))
    a = check(z, x)
    assert torch.equal(a, ds.process_logits(z.cuda(), **dev(x)))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    V, R = 1 << 24, 1
    B = 131                                                            # B V > 2^31 entries
    z = torch.zeros(B, V, dtype=torch.bfloat16, device="cuda")
    z[B - 1, V - 1] = 3.0
    h = torch.full((B, 2), V - 1, dtype=torch.int32, device="cuda")
    out = ds.process_logits(z, history=h, repetition=torch.full((B,), 2.0, device="cuda"),
                            frequency=torch.full((B,), 0.25, device="cuda"))
    assert float(out[B - 1, V - 1]) == 1.0 and float(out[B - 1, V - 2]) == 0.0 and float(out[0, V - 1]) == -0.5


@pytest.mark.gpu
def test_captured_graph_and_another_stream():
    z, x = make(4, 2, 7001, 200, seed=61, nb=4, masked=2)
    zc, xc = z.cuda(), dev(x)
    want = ds.process_logits(zc, **xc)
    s = torch.cuda.Stream()
    plan = ds.ProcessPlan(zc, stream=s, **xc)
    out = plan.run()
    s.synchronize()
    assert torch.equal(out, want)
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            plan.run(s)
    zc.mul_(0.5)
    xc["lengths"].clamp_(max=17)
    xc["prompt_lengths"].clamp_(max=5)
    out.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ds.process_logits(zc, **xc))


@pytest.mark.gpu
def test_processed_targets_are_verified():
    """A whole round: bf16 target logits under each request's tools, the drafted tokens counted, into verify."""
    from oracle import oracle
    B, G, V = 6, 5, 4001
    z, x = make(B, G + 1, V, 120, seed=71, dtype=torch.bfloat16, nb=4, masked=3)
    g = torch.Generator().manual_seed(3)
    tok = torch.randint(0, V, (B, G), generator=g, dtype=torch.int32)
    x["drafted"] = tok
    d = torch.randn(B, G, V, generator=g) * 2
    q = ds.process_logits(z.cuda(), dtype=torch.float32, **dev(x))
    n, out = ds.verify(d.cuda(), q, tok.cuda(), seed=5)
    ref = oracle.verify(gamma=G, T=1.0, seed=5, draft_logits=d.numpy(), target_logits=q.cpu().numpy(),
                        draft_tokens=tok.numpy())
    assert (n.cpu().numpy() == ref.n_accepted).all()
    ok = allowed_rows(x, B * (G + 1), V).view(B, G + 1, V)
    for b in range(B):
        for k in range(int(n[b]) + 1):
            assert ok[b, k, int(out[b, k])]                          # no masked token is accepted or drawn
