"""Operators around the logits of a speculative block, as cases to time.

* ``process`` / ``process_grad``: what a request asks of its logits before they are verified, sampled
  or trained on: penalties for tokens that its text already holds, biases, a grammar's mask; and the
  gradient with respect to the raw logits;
* ``distill`` / ``distill_grad``: the loss of a row of logits against a teacher's K largest log
  probabilities (relative entropy and L1 distance over those K and the rest), with its gradient in the
  same call or without it, and the gradient alone from what the forward call left.

gamma + 1 = 8 rows of a request are a verified block, gamma = 7 a training block.  Every case runs
either in a plain form (elementary operations in 32 bits) or through the entry points of
``semi_autoregressive_drafting_gb300``.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the target's logits of one request's verified block, in the midst of a conversation: latency
        dict(name="process_one_request", kind="process", B=1, R=8, V=151936, dtype="bf16", out="f32", H=2048,
             bias=0, masked=0.0, pad=0),
        # the same for a batch of 64, with the few dozen biases that a client may send
        dict(name="process_batch", kind="process", B=64, R=8, V=151936, dtype="bf16", out="f32", H=8192,
             bias=32, masked=0.0, pad=0),
        # decoding one token for each of 512 requests, three quarters of them under a grammar
        dict(name="process_grammar", kind="process", B=512, R=1, V=151936, dtype="f32", out="f32", H=1024,
             bias=0, masked=0.75, pad=0),
        # a few requests with very long texts, one token each, the largest vocabulary
        dict(name="process_long", kind="process", B=8, R=1, V=262144, dtype="bf16", out="bf16", H=131072,
             bias=300, masked=0.25, pad=0),
        # training under the processors that decoding applied: an odd vocabulary in padded rows
        dict(name="process_grad_odd", kind="process_grad", B=77, R=7, V=50021, dtype="f32", out="f32", H=1023,
             masked=0.5, pad=27),
        # the same at the largest batch and vocabulary, in bf16
        dict(name="process_grad_train", kind="process_grad", B=512, R=7, V=262144, dtype="bf16", out="bf16",
             H=2048, masked=0.25, pad=0),
        # distilling one request's block: loss and gradient, the teacher's twenty most likely tokens
        dict(name="distill_one_request", kind="distill", N=7, V=151936, dtype="bf16", K=20, T=1.0, kl=1.0, l1=0.0,
             rest=True, grad=True, pad=0),
        # 64 requests, fp32, the L1 distance that acceptance depends on beside the relative entropy
        dict(name="distill_batch", kind="distill", N=448, V=151936, dtype="f32", K=32, T=1.0, kl=0.1, l1=0.9,
             rest=True, grad=True, pad=0),
        # the training step at the largest batch and vocabulary
        dict(name="distill_train", kind="distill", N=3584, V=262144, dtype="bf16", K=64, T=1.0, kl=1.0, l1=0.0,
             rest=True, grad=True, pad=0),
        # validation: the loss alone, an odd vocabulary in padded rows, a temperature, the rest left out
        dict(name="distill_validate_odd", kind="distill", N=499, V=50021, dtype="f32", K=50, T=0.7, kl=1.0, l1=0.0,
             rest=False, grad=False, pad=27),
        # the gradient alone, for a loss whose weights are known after the forward pass
        dict(name="distill_grad_batch", kind="distill_grad", N=448, V=151936, dtype="f32", K=32, T=1.0, kl=0.1,
             l1=0.9, rest=True, pad=0),
        # the same at the largest batch, in bf16
        dict(name="distill_grad_train", kind="distill_grad", N=3584, V=262144, dtype="bf16", K=64, T=1.0, kl=1.0,
             l1=0.0, rest=True, pad=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["process", "process", "process", "process_grad", "distill", "distill", "distill_grad"])
    dtype = rng.choice(["f32", "bf16"])
    V = _log_int(rng, 1000, 262144)
    pad = rng.choice([0, 0, 1, 24, 37])
    size = 1 if dtype == "bf16" else 2
    if kind in ("process", "process_grad"):
        R = rng.choice([1, 1, 2, 5, 7, 8])
        most = 64 * 8 * 151936 if kind == "process" else 3584 * 262144 // size
        B = _log_int(rng, 1, max(1, min(512, most // (R * V))))
        c = dict(kind=kind, B=B, R=R, V=V, dtype=dtype, out=rng.choice([dtype, "f32"]),
                 H=_log_int(rng, 1, max(1, min(131072, (1 << 20) // B))),
                 masked=rng.choice([0.0, 0.3, 1.0]), pad=pad)
        if kind == "process":
            c["bias"] = rng.choice([0, 0, 3, 40, 300])
        return c
    N = _log_int(rng, 1, max(1, min(3584, 3584 * 262144 // (V * size))))
    kl, l1 = rng.choice([(1.0, 0.0), (1.0, 0.0), (0.1, 0.9), (0.0, 1.0)]) if N <= 512 else (1.0, 0.0)
    c = dict(kind=kind, N=N, V=V, dtype=dtype, K=rng.choice([1, 5, 20, 32, 50, 64, 100, 128]),
             T=rng.choice([1.0, 1.0, 0.7, 2.0]), kl=kl, l1=l1, rest=rng.random() < 0.75, pad=pad)
    if kind == "distill":
        c["grad"] = rng.random() < 0.7
    return c


# ------------------------------------------------------------------ inputs
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 29)
    return gen


def _normal(gen, N, V, pad, std, dtype):
    """N(0, std^2) rows of V + pad entries on the GPU, drawn in fp32 some rows at a time; the first V."""
    out = torch.empty(N, V + pad, dtype=dtype, device="cuda")
    step = max(1, (1 << 27) // (V + pad))
    for i in range(0, N, step):
        n = min(step, N - i)
        out[i:i + n] = torch.randn(n, V + pad, generator=gen, device="cuda") * std
    return out[:, :V]


def _text(gen, shape, V):
    """Tokens as text has them: a rank's frequency falls as 1 / rank, the ids shuffled."""
    u = torch.rand(shape, generator=gen, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
    return torch.randperm(V, generator=gen, device="cuda")[rank].to(torch.int32)


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda")


def _process_inputs(case, seed):
    gen = _gen(case, seed)
    B, R, V, H = case["B"], case["R"], case["V"], case["H"]
    x = dict(z=_normal(gen, B * R, V, case["pad"], 3.0, _DT[case["dtype"]]).unflatten(0, (B, R)))
    # texts of any length up to H, the first part of each the prompt
    x["history"] = _text(gen, (B, H), V)
    x["lengths"] = (_rand(gen, B) * (H + 1)).to(torch.int32).clamp_(max=H)
    x["prompts"] = (_rand(gen, B) * x["lengths"]).to(torch.int32)
    # half of the drafted tokens are in the text already; some requests' blocks are shorter
    again = x["history"].gather(1, torch.randint(0, H, (B, R - 1), generator=gen, device="cuda"))
    x["drafted"] = torch.where(_rand(gen, B, R - 1) < 0.5, again, _text(gen, (B, R - 1), V))
    short = 1 + (_rand(gen, B) * 3 * R).long()
    x["drafted"][torch.arange(R - 1, device="cuda")[None] >= short[:, None]] = -1
    # one request in five asks for no penalty
    some = _rand(gen, B) < 0.8
    x["repetition"] = torch.where(some, 1.0 + 0.3 * _rand(gen, B), 1.0)
    x["presence"] = torch.where(some, _rand(gen, B), 0.0)
    x["frequency"] = torch.where(some, 0.5 * _rand(gen, B), 0.0)
    nb = case.get("bias", 0)
    if nb:
        x["bias_tokens"] = _text(gen, (B, nb), V)
        used = (_rand(gen, B) * (nb + 1)).long()
        x["bias_tokens"][torch.arange(nb, device="cuda")[None] >= used[:, None]] = -1
        x["bias"] = 4.0 * torch.randn(B, nb, generator=gen, device="cuda")
    if case["masked"]:
        # masks of a grammar's states, which rows share: half of them strict, half with little ruled out
        M, W = min(B * R, 256), (V + 31) // 32
        words = torch.empty(M, W, dtype=torch.int32, device="cuda")
        weight = (torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda"))
        for i in range(0, M, 32):
            n = min(32, M - i)
            share = torch.where(torch.arange(i, i + n, device="cuda") % 2 == 0, 0.005, 0.9)
            bits = _rand(gen, n, W * 32) < share[:, None]
            word = (bits.view(n, W, 32) * weight).sum(-1)
            words[i:i + n] = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
        rows = torch.randint(0, M, (B, R), generator=gen, device="cuda", dtype=torch.int32)
        x["mask"], x["mask_rows"] = words, torch.where(_rand(gen, B, 1) < case["masked"], rows, -1)
    if case["kind"] == "process_grad":
        x["grad"] = _normal(gen, B * R, V, 0, 1e-3, _DT[case["out"]]).unflatten(0, (B, R))
    return x


def _distill_inputs(case, seed):
    gen = _gen(case, seed)
    N, V, K, T = case["N"], case["V"], case["K"], case["T"]
    dt = _DT[case["dtype"]]
    x = dict(z=_normal(gen, N, V, case["pad"], 3.0, dt))
    # K different tokens a row; the teacher's probabilities fall as a power of the rank and hold most of it
    first = torch.randint(0, V, (N, 1), generator=gen, device="cuda")
    stride = 1 + (_rand(gen, N, 1) * (V // K - 1)).long()
    ids = (first + stride * torch.arange(K, device="cuda")) % V
    power = 0.8 + 1.5 * _rand(gen, N, 1)
    q = torch.arange(1, K + 1, device="cuda").double()[None] ** -power.double()
    q = q / q.sum(1, keepdim=True) * (0.75 + 0.24 * _rand(gen, N, 1).double())
    # a trained student: its probabilities are within a factor of the teacher's, and not next to them
    off = (0.15 + 1.0 * _rand(gen, N, K)) * torch.where(_rand(gen, N, K) < 0.5, 1.0, -1.0)
    off = torch.where(((q * off.exp()).sum(1, keepdim=True) > 0.98), -off.abs(), off).double()
    p = q * off.exp()
    step = max(1, (1 << 26) // V)
    for i in range(0, N, step):
        zi = x["z"][i:i + step].float() / T
        zi.scatter_(1, ids[i:i + step], float("-inf"))
        base = torch.logsumexp(zi, dim=1, keepdim=True).double()
        pi = p[i:i + step]
        lift = T * (pi.log() - (1.0 - pi.sum(1, keepdim=True)).log() + base)
        x["z"][i:i + step].scatter_(1, ids[i:i + step], lift.to(dt))
    # one row in five has fewer entries (a teacher cut at a share of its mass): padded with -1
    cut = torch.where(_rand(gen, N) < 0.2, 1 + (_rand(gen, N) * K).long(), K)
    none = torch.arange(K, device="cuda")[None] >= cut[:, None]
    x["ids"] = torch.where(none, -1, ids).to(torch.int32)
    x["logq"] = torch.where(none, float("-inf"), q.log().float())
    # the positions' weights of a block of seven; a few rows are padding
    x["weight"] = torch.exp(-(torch.arange(N, device="cuda") % 7).float() / 7.0) / N
    if N >= 16:
        x["weight"][_rand(gen, N) < 0.03] = 0.0
    if case["kind"] == "distill_grad":
        x["norm"] = torch.empty(N, 4, device="cuda")
        for i in range(0, N, step):
            zi = x["z"][i:i + step].double()
            idi = x["ids"][i:i + step].long()
            at = torch.where(idi >= 0, idi, idi[:, :1])
            others = zi.clone().scatter_(1, at, float("-inf"))
            for j, s in ((0, zi), (2, others)):
                m = s.amax(1)
                x["norm"][i:i + step, j] = m
                x["norm"][i:i + step, j + 1] = ((s - m[:, None]) / T).exp().sum(1).log()
    return x


def _inputs(case, seed):
    return _process_inputs(case, seed) if case["kind"].startswith("process") else _distill_inputs(case, seed)


def prepare(case, seed):
    x = _inputs(case, seed)
    state = dict(case=case, **x)
    if own:
        import semi_autoregressive_drafting_gb300 as ds
        kind = case["kind"]
        if kind == "process":
            state["plan"] = ds.ProcessPlan(
                x["z"], history=x["history"], lengths=x["lengths"], prompt_lengths=x["prompts"],
                drafted=x["drafted"], repetition=x["repetition"], presence=x["presence"], frequency=x["frequency"],
                bias_tokens=x.get("bias_tokens"), bias=x.get("bias"), mask=x.get("mask"),
                mask_rows=x.get("mask_rows"), dtype=_DT[case["out"]])
        elif kind == "process_grad":
            state["plan"] = ds.ProcessGradPlan(
                x["grad"], x["z"], history=x["history"], lengths=x["lengths"], prompt_lengths=x["prompts"],
                drafted=x["drafted"], repetition=x["repetition"], mask=x.get("mask"), mask_rows=x.get("mask_rows"))
        else:
            how = dict(T=case["T"], alpha=(case["kl"], case["l1"]), rest=case["rest"])
            if kind == "distill":
                state["plan"] = ds.DistillPlan(x["z"], x["ids"], x["logq"], weight=x["weight"],
                                               want_grad=case["grad"], **how)
            else:
                state["plan"] = ds.DistillGradPlan(x["z"], x["ids"], x["logq"], x["norm"], x["weight"], **how)
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    kind = state["case"]["kind"]
    if own:
        o = state["plan"].run()
        if kind == "distill":
            res = dict(loss=o.loss, parts=o.parts, norm=o.norm)
            if state["case"]["grad"]:
                res["grad"] = o.grad_logits
            return res
        return o
    return _PLAIN[kind](state)


def _allowed(s):
    """Which entries the rows' masks leave [B, R, V], or None."""
    if s.get("mask") is None:
        return None
    B, R, V = s["z"].shape
    rows = s["mask_rows"].long()
    words = s["mask"][rows.clamp(min=0)]
    bits = (words[..., None] >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1
    return (bits.view(B, R, -1)[..., :V] == 1) | (rows < 0)[..., None]


def _counts(s):
    """How often each row's request has generated each token [B, R, V], and whether its text holds it."""
    B, R, V = s["z"].shape
    tok, dev = s["history"].long(), s["z"].device
    at = torch.arange(tok.shape[1], device=dev)[None]
    used = (at < s["lengths"][:, None]) & (tok >= 0)
    made = used & (at >= s["prompts"][:, None])
    count = torch.zeros(B, V + 1, device=dev)
    count.scatter_add_(1, torch.where(made, tok, V), torch.ones_like(tok, dtype=torch.float32))
    seen = torch.zeros(B, V + 1, dtype=torch.bool, device=dev)
    seen.scatter_(1, torch.where(used, tok, V), True)
    # row k counts the k tokens drafted before it
    k = torch.arange(R, device=dev)
    tok = s["drafted"].long()[:, None, :].expand(B, R, R - 1)
    tok = torch.where((k[None, :R - 1] < k[:, None]) & (tok >= 0), tok, V)
    count = count[:, None, :].repeat(1, R, 1).scatter_add_(2, tok, torch.ones_like(tok, dtype=torch.float32))
    seen = seen[:, None, :].repeat(1, R, 1).scatter_(2, tok, True)
    return count[..., :V], seen[..., :V]


def _per_request(x):
    return x[:, None, None]


def _plain_process(s):
    z = s["z"].float()
    count, seen = _counts(s)
    rep = _per_request(s["repetition"])
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - _per_request(s["frequency"]) * count - _per_request(s["presence"]) * (count > 0)
    if s.get("bias") is not None:
        B, V = z.shape[0], z.shape[2]
        add = torch.zeros(B, V + 1, device=z.device)
        tok = s["bias_tokens"].long()
        add.scatter_add_(1, torch.where(tok >= 0, tok, V), s["bias"])
        z = z + add[:, None, :V]
    ok = _allowed(s)
    if ok is not None:
        z = torch.where(ok, z, float("-inf"))
    return z.to(_DT[s["case"]["out"]])


def _plain_process_grad(s):
    _, seen = _counts(s)
    rep = _per_request(s["repetition"])
    g = s["grad"].float()
    g = torch.where(seen, torch.where(s["z"] > 0, g / rep, g * rep), g)
    ok = _allowed(s)
    if ok is not None:
        g = torch.where(ok, g, 0.0)
    return g.to(s["z"].dtype)


def _outcomes(s, z, norm):
    """The K + 1 outcomes in 64 bits: teacher's and student's probabilities [N, K + 1], their logs, and
    which count; the last one is the rest."""
    c, T = s["case"], s["case"]["T"]
    ids = s["ids"].long()
    given = ids >= 0
    zs = z.gather(1, ids.clamp(min=0)).double()
    norm = norm.double()
    lnp = torch.where(given, (zs - norm[:, :1]) / T - norm[:, 1:2], float("-inf"))
    lnp_rest = (norm[:, 2:3] - norm[:, :1]) / T + norm[:, 3:] - norm[:, 1:2]
    logq = torch.where(given, s["logq"].double(), float("-inf"))
    q_rest = (1.0 - logq.exp().sum(1, keepdim=True)).clamp(min=0.0)
    lnp = torch.cat([lnp, lnp_rest], dim=1)
    logq = torch.cat([logq, q_rest.log()], dim=1)
    count = torch.cat([given, torch.full_like(given[:, :1], c["rest"])], dim=1)
    return logq.exp(), logq, lnp.exp(), lnp, count


def _plain_gradient(s, z, norm):
    c, T = s["case"], s["case"]["T"]
    q, _, p, _, count = _outcomes(s, z, norm)
    # p times the derivative of the loss with respect to each outcome's probability
    pd = torch.where(count, -c["kl"] * q + c["l1"] * p * torch.sign(p - q), 0.0)
    mean = pd.sum(1, keepdim=True)
    part = (pd - p * mean) / T * s["weight"].double()[:, None]
    # the rest's share goes to its entries by their probability within it
    g = ((z - norm[:, 2:3]) / T - norm[:, 3:]).exp() * part[:, -1:].float()
    g = torch.cat([g, g[:, :1]], dim=1)  # (a last column for rows' missing entries)
    ids = s["ids"].long()
    g.scatter_(1, torch.where(ids >= 0, ids, z.shape[1]), part[:, :-1].float())
    return g[:, :z.shape[1]].to(s["z"].dtype)


def _normaliser(z, T):
    m = z.amax(1)
    return torch.stack([m, ((z - m[:, None]) / T).exp().sum(1).log()], dim=1)


def _plain_distill(s):
    c = s["case"]
    z, ids = s["z"].float(), s["ids"].long()
    others = torch.cat([z, z[:, :1]], dim=1)
    others.scatter_(1, torch.where(ids >= 0, ids, z.shape[1]), float("-inf"))
    norm = torch.cat([_normaliser(z, c["T"]), _normaliser(others[:, :z.shape[1]], c["T"])], dim=1)
    q, logq, p, lnp, count = _outcomes(s, z, norm)
    kl = torch.where(count & (q > 0), q * (logq - lnp), 0.0).sum(1)
    l1 = torch.where(count, (p - q).abs(), 0.0).sum(1)
    on = s["weight"] != 0
    res = dict(loss=torch.where(on, s["weight"] * (c["kl"] * kl + c["l1"] * l1), 0.0).float(),
               parts=torch.where(on[:, None], torch.stack([kl, l1], dim=1), 0.0).float(),
               norm=torch.where(on[:, None], norm, 0.0))
    if c["grad"]:
        res["grad"] = _plain_gradient(s, z, norm)
    return res


def _plain_distill_grad(s):
    return _plain_gradient(s, s["z"].float(), s["norm"])


_PLAIN = dict(process=_plain_process, process_grad=_plain_process_grad, distill=_plain_distill,
              distill_grad=_plain_distill_grad)


# ------------------------------------------------------------------ work
def work(case):
    es = {"f32": 4, "bf16": 2}
    V = case["V"]
    if case["kind"].startswith("process"):
        N, B = case["B"] * case["R"], case["B"]
        # a masked entry's value is not needed: constrained rows keep (0.005 + 0.9) / 2 of theirs
        kept = 1.0 - case["masked"] * (1.0 - 0.4525)
        small = B * case["H"] // 2 * 4 + B * 20 + B * (case["R"] - 1) * 4 + B * case.get("bias", 0) * 8
        small += int(N * case["masked"]) * V // 8 + N * 4
        if case["kind"] == "process":
            return {"bytes": int(N * V * (kept * es[case["dtype"]] + es[case["out"]])) + small, "flops": N * V}
        # raw logits decide the gradient only where a text holds their token
        raw = min(N * V, N * case["H"] // 4) * es[case["dtype"]]
        return {"bytes": int(N * V * (kept * es[case["out"]] + es[case["dtype"]])) + raw + small, "flops": N * V}
    N = case["N"]
    size = N * V * es[case["dtype"]]
    small = N * case["K"] * 8 + N * 32
    if case["kind"] == "distill":
        return {"bytes": size * (2 if case["grad"] else 1) + small, "flops": (9 if case["grad"] else 5) * N * V}
    return {"bytes": 2 * size + small, "flops": 4 * N * V}


# ------------------------------------------------------------------ in 64 bits
def _keep(t, N, V):
    """Results of the largest cases are kept in 32 bits: in 64 they would not be worth their memory."""
    return t.float() if N * V > 1 << 28 else t


def _exact_process(case, x):
    B, R, V = case["B"], case["R"], case["V"]
    dev = x["z"].device
    b = torch.arange(B, device=dev)[:, None].expand(B, case["H"])
    spot = torch.arange(case["H"], device=dev).expand(B, case["H"])
    inside = spot < x["lengths"][:, None]
    made = inside & (spot >= x["prompts"][:, None])
    flat = b * V + x["history"]
    count = torch.bincount(flat[made], minlength=B * V).view(B, V)
    text = torch.bincount(flat[inside], minlength=B * V).view(B, V)
    shift = torch.zeros(B, V, dtype=torch.float64, device=dev)
    if x.get("bias") is not None:
        for j in range(x["bias"].shape[1]):
            t = x["bias_tokens"][:, j].long()
            who = torch.nonzero(t >= 0)[:, 0]
            shift[who, t[who]] += x["bias"][who, j].double()
    forward = case["kind"] == "process"
    out = []
    for r in range(R):
        if r:
            t = x["drafted"][:, r - 1].long()
            who = torch.nonzero(t >= 0)[:, 0]
            count[who, t[who]] += 1
            text[who, t[who]] += 1
        z = x["z"][:, r].double()
        rep = x["repetition"].double()[:, None]
        scale = torch.where(text > 0, torch.where(z > 0, 1.0 / rep, rep), 1.0)
        if forward:
            y = z * scale - x["frequency"].double()[:, None] * count - x["presence"].double()[:, None] * count.clamp(max=1)
            y += shift
        else:
            y = x["grad"][:, r].double() * scale
        if x.get("mask") is not None:
            v = torch.arange(V, device=dev)
            row = x["mask_rows"][:, r].long()
            who = torch.nonzero(row >= 0)[:, 0]
            bit = torch.bitwise_right_shift(x["mask"][row[who]].long()[:, v // 32], v % 32) % 2
            y[who] = y[who].masked_fill(bit == 0, -math.inf if forward else 0.0)
        out.append(_keep(y, B * R, V))
    return torch.stack(out, dim=1)


def _exact_distill(case, x):
    """By automatic differentiation of the loss."""
    N, V, T = case["N"], case["V"], case["T"]
    parts = []
    want = case["kind"] == "distill_grad" or case["grad"]
    step = max(1, (1 << 25) // V)
    for i in range(0, N, step):
        z = x["z"][i:i + step].double().requires_grad_(want)
        ids, lq = x["ids"][i:i + step].long(), x["logq"][i:i + step].double()
        w = x["weight"][i:i + step].double()
        n = z.shape[0]
        row, col = torch.nonzero(ids >= 0, as_tuple=True)
        with torch.set_grad_enabled(want):
            lp = torch.log_softmax(z / T, dim=1)
            hot = torch.zeros_like(lp, dtype=torch.bool)
            hot[row, ids[row, col]] = True
            rest = torch.logsumexp(lp.masked_fill(hot, -math.inf), dim=1)
            a, b = lq[row, col], lp[row, ids[row, col]]
            zero = torch.zeros(n, dtype=torch.float64, device=z.device)
            kl = zero.index_add(0, row, a.exp() * (a - b))
            l1 = zero.index_add(0, row, (a.exp() - b.exp()).abs())
            left = (1.0 - zero.index_add(0, row, a.exp())).clamp(min=0.0)
            if case["rest"]:
                kl = kl + torch.special.xlogy(left, left) - left * rest
                l1 = l1 + (left - rest.exp()).abs()
            loss = w * (case["kl"] * kl + case["l1"] * l1)
        one = {}
        if case["kind"] == "distill":
            keep = (w != 0).double()
            zd = z.detach()
            zo = zd.masked_fill(hot, -math.inf)
            m, mo = zd.amax(1), zo.amax(1)
            norm = torch.stack([m, torch.logsumexp((zd - m[:, None]) / T, 1), mo,
                                torch.logsumexp((zo - mo[:, None]) / T, 1)], dim=1)
            one = dict(loss=loss.detach(), parts=torch.stack([kl, l1], dim=1).detach() * keep[:, None],
                       norm=norm * keep[:, None])
        if want:
            one["grad"] = _keep(torch.autograd.grad(loss.sum(), z)[0], N, V)
        parts.append(one)
    res = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    return res if case["kind"] == "distill" else res["grad"]


def exact(case, seed):
    x = _inputs(case, seed)
    return _exact_process(case, x) if case["kind"].startswith("process") else _exact_distill(case, x)
