"""The language-model operators around the Markov head's training and scoring, as cases to time.

Three operators and their gradients, in the order in which one training step of the head meets
them (gamma positions of B requests are N = B * gamma rows):

* ``embed`` / ``embed_grad``: rows of the head's table for the conditioning tokens, scaled, and
  the table's gradient, the sum of every token's rows;
* ``bias_grad``: the gradient of the low-rank bias product B_k = a W2, that is
  grad_a = G W2 and grad_W2 = G^T a for gradients G of the logits;
* ``logprob`` / ``logprob_grad``: log probability, entropy, rank and top alternatives of given
  tokens under softmax(z / T), and the gradient of the first two with respect to z.

Every case runs either in a plain form (elementary operations in 32 bits) or through the entry
points of ``semi_autoregressive_drafting_gb300``.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # scoring the verified block of one request while serving: gamma + 1 = 8 rows of target
        # logits, the usual five alternatives; latency is what counts
        dict(name="logprob_one_request", kind="logprob", N=8, V=151936, dtype="bf16", T=1.0, top=5,
             pad=0, masked=False),
        # the same for a batch of 64 requests in fp32, with the most alternatives that servers offer
        dict(name="logprob_batch", kind="logprob", N=512, V=151936, dtype="f32", T=1.0, top=20, pad=0,
             masked=False),
        # an odd vocabulary in rows padded to a common stride, some entries switched off by a
        # sampling mask, a temperature
        dict(name="logprob_masked_odd", kind="logprob", N=77, V=50021, dtype="f32", T=0.7, top=8, pad=27,
             masked=True),
        # the training forward pass at the largest batch and vocabulary: 512 * 7 rows, no alternatives
        dict(name="logprob_train", kind="logprob", N=3584, V=262144, dtype="bf16", T=1.0, top=0, pad=0,
             masked=False),
        # the gradient with respect to fp32 logits for 64 requests of a block of 7
        dict(name="logprob_grad_batch", kind="logprob_grad", N=448, V=151936, dtype="f32", T=1.0),
        # the same at the largest batch, in bf16
        dict(name="logprob_grad_train", kind="logprob_grad", N=3584, V=262144, dtype="bf16", T=1.0),
        # the conditioning rows of one request's block, W1[x_{k-1}]
        dict(name="embed_one_request", kind="embed", N=8, V=151936, D=256, dtype="bf16", scale=1.0),
        # a backbone's input embeddings of a training batch, scaled by sqrt(d)
        dict(name="embed_train", kind="embed", N=32768, V=151936, D=4096, dtype="bf16", scale=64.0),
        # the gradient of W1 for 64 requests of a block of 7, tokens as text has them
        dict(name="embed_grad_batch", kind="embed_grad", N=448, V=151936, D=256, dtype="f32", scale=1.0),
        # the gradient of a backbone's table for a training batch in bf16
        dict(name="embed_grad_train", kind="embed_grad", N=32768, V=151936, D=2560, dtype="bf16",
             scale=math.sqrt(2560.0)),
        # the bias product's gradients for 64 requests of a block of 7, from the fp32 gradient
        # that the training loss writes
        dict(name="bias_grad_batch", kind="bias_grad", N=448, V=151936, r=256, dtype="f32",
             weights="bf16", layout="vr"),
        # the same for 512 requests and the largest vocabulary, from a bf16 gradient
        dict(name="bias_grad_train", kind="bias_grad", N=3584, V=262144, r=256, dtype="bf16",
             weights="bf16", layout="vr"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["logprob", "logprob", "logprob_grad", "embed", "embed_grad", "bias_grad", "bias_grad"])
    dtype = rng.choice(["f32", "bf16"])
    T = rng.choice([1.0, 1.0, 0.6, 0.8, 1.3])
    if kind in ("logprob", "logprob_grad"):
        V = _log_int(rng, 1000, 262144)
        N = _log_int(rng, 1, max(1, min(3584, 3584 * 262144 // V // (1 if dtype == "bf16" else 2))))
        c = dict(kind=kind, N=N, V=V, dtype=dtype, T=T)
        if kind == "logprob":
            # the plain form ranks whole rows: alternatives up to the batch size that asks for them
            top = rng.choice([0, 1, 5, 20, 32]) if N * V <= 512 * 151936 else 0
            c.update(top=top, pad=rng.choice([0, 0, 1, 24, 37]), masked=rng.random() < 0.3)
        return c
    if kind in ("embed", "embed_grad"):
        V = _log_int(rng, 1000, 262144)
        D = rng.choice([64, 256, 250, 512, 1000, 1023, 2560, 4096])
        top = 32768 * 4096 if kind == "embed" else 32768 * 2560
        N = _log_int(rng, 1, max(1, min(65536, top // D)))
        if kind == "embed_grad":
            V = min(V, 151936 * 2560 // D)
        return dict(kind=kind, N=N, V=V, D=D, dtype=dtype,
                    scale=rng.choice([1.0, 0.5, math.sqrt(float(D))]))
    if rng.random() < 0.25:  # a small head trained in fp32
        V = _log_int(rng, 512, 8192)
        return dict(kind=kind, N=_log_int(rng, 1, 256), V=V, r=8 * rng.randint(1, 16), dtype="f32",
                    weights="f32", layout=rng.choice(["vr", "rv"]))
    V = _log_int(rng, 4096, 262144)
    r = rng.choice([64, 64, 72, 128, 200, 256, 256, 512])
    N = _log_int(rng, 1, max(1, min(3584, 3584 * 262144 * 256 // (V * r) // (1 if dtype == "bf16" else 2))))
    return dict(kind=kind, N=N, V=V, r=r, dtype=dtype, weights="bf16", layout=rng.choice(["vr", "rv"]))


# ------------------------------------------------------------------ inputs
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _normal(gen, shape, std, dtype):
    """N(0, std^2) on the GPU, drawn in fp32 some rows at a time."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 27) // max(1, shape[1]))
    for i in range(0, shape[0], step):
        n = min(step, shape[0] - i)
        out[i:i + n] = torch.randn(n, shape[1], generator=gen, device="cuda") * std
    return out


def _text_tokens(gen, N, V):
    """Tokens as text has them: a rank's frequency falls as 1 / rank, the ids shuffled."""
    u = torch.rand(N, generator=gen, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
    return torch.randperm(V, generator=gen, device="cuda")[rank].to(torch.int32)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 17)
    k, N, V = case["kind"], case["N"], case["V"]
    dt = _DT[case["dtype"]]
    if k in ("logprob", "logprob_grad"):
        pad = case.get("pad", 0)
        z = _normal(gen, (N, V + pad), 3.0, dt)[:, :V]
        tok = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
        if case.get("masked"):
            # one entry in eight switched off, by -inf or by the lowest finite number; never the
            # given token
            off = torch.rand(N, V, generator=gen, device="cuda")
            off.scatter_(1, tok.long()[:, None], 1.0)
            z.masked_fill_(off < 0.0625, float("-inf"))
            z.masked_fill_((off >= 0.0625) & (off < 0.125), torch.finfo(dt).min)
        else:
            # a trained model's rows: the given token is often among the likely ones
            lift = 4.0 * torch.rand(N, generator=gen, device="cuda")
            z[torch.arange(N, device="cuda"), tok.long()] += lift.to(dt)
        x = dict(z=z, tok=tok)
        if k == "logprob_grad":
            x["g_logp"] = torch.randn(N, generator=gen, device="cuda")
            x["g_ent"] = 0.01 * torch.randn(N, generator=gen, device="cuda")
            # what the forward pass left: the rows' largest logit, the log of the sum of
            # exponentials above it, and the entropy
            norm = torch.empty(N, 2, device="cuda")
            ent = torch.empty(N, device="cuda")
            step = max(1, (1 << 26) // V)
            for i in range(0, N, step):
                zi = z[i:i + step].double()
                m = zi.max(dim=1).values
                d = (zi - m[:, None]) / case["T"]
                e = d.exp()
                s = e.sum(dim=1)
                norm[i:i + step, 0] = m
                norm[i:i + step, 1] = s.log()
                ent[i:i + step] = s.log() - (e * d).sum(dim=1) / s
            x.update(norm=norm, entropy=ent)
        return x
    if k == "embed":
        D = case["D"]
        tok = _text_tokens(gen, N, V)
        if N >= 16:
            tok[torch.rand(N, generator=gen, device="cuda") < 0.03] = -1  # padding of ragged sequences
        return dict(W=_normal(gen, (V, D), 0.02, dt), tok=tok)
    if k == "embed_grad":
        D = case["D"]
        tok = _text_tokens(gen, N, V)
        if N >= 16:
            tok[torch.rand(N, generator=gen, device="cuda") < 0.03] = -1
        return dict(g=_normal(gen, (N, D), 1.0, dt), tok=tok)
    if k == "bias_grad":
        r, wdt = case["r"], _DT[case["weights"]]
        # gradients of a cross entropy: small everywhere, minus one at the label
        G = _normal(gen, (N, V), 1e-3, dt)
        lab = torch.randint(0, V, (N,), generator=gen, device="cuda")
        G[torch.arange(N, device="cuda"), lab] = -1.0
        a = _normal(gen, (N, r), 0.02, wdt)
        W2 = _normal(gen, (V, r) if case["layout"] == "vr" else (r, V), 0.02, wdt)
        return dict(G=G, a=a, W2=W2)
    raise ValueError(k)


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if own:
        import semi_autoregressive_drafting_gb300 as ds
        k, x = case["kind"], state
        if k == "logprob":
            state["plan"] = ds.LogprobPlan(x["z"], x["tok"], T=case["T"], top=case["top"])
        elif k == "logprob_grad":
            state["plan"] = ds.LogprobGradPlan(x["z"], x["tok"], x["norm"], T=case["T"],
                                               grad_logp=x["g_logp"], grad_entropy=x["g_ent"],
                                               entropy=x["entropy"])
        elif k == "embed":
            state["plan"] = ds.EmbeddingPlan(x["W"], x["tok"], scale=case["scale"])
        elif k == "embed_grad":
            state["plan"] = ds.EmbeddingGradPlan(x["g"], x["tok"], case["V"], scale=case["scale"])
        else:
            state["plan"] = ds.BiasGradPlan(x["G"], x["a"], x["W2"], w2_layout=case["layout"])
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    k = state["case"]["kind"]
    if own:
        o = state["plan"].run()
        if k == "logprob":
            res = dict(logp=o.logp, norm=o.norm, entropy=o.entropy, rank=o.rank)
            if state["case"]["top"]:
                res.update(top_ids=o.top_ids, top_logp=o.top_logp)
            return res
        if k == "bias_grad":
            return dict(grad_a=o[0], grad_W2=o[1])
        return o
    return _PLAIN[k](state)


def _plain_logprob(s):
    c = s["case"]
    z, tok = s["z"].float(), s["tok"].long()
    m = z.max(dim=1).values
    d = (z - m[:, None]) / c["T"]
    e = d.exp()
    total = e.sum(dim=1)
    logsum = total.log()
    zx = z.gather(1, tok[:, None])
    res = dict(logp=(zx[:, 0] - m) / c["T"] - logsum, norm=torch.stack([m, logsum], dim=1),
               entropy=logsum - torch.where(e > 0, e * d, 0.0).sum(dim=1) / total,
               rank=((z > zx).sum(dim=1) + 1).to(torch.int32))
    if c["top"]:
        # whole-number keys in the order of (logit, then the lower index): no two are equal
        bits = (z + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        key = order * (1 << 25) - torch.arange(c["V"], device=z.device)
        ids = key.topk(c["top"], dim=1).indices
        res.update(top_ids=ids.to(torch.int32),
                   top_logp=(z.gather(1, ids) - m[:, None]) / c["T"] - logsum[:, None])
    return res


def _plain_logprob_grad(s):
    c = s["case"]
    z, tok = s["z"].float(), s["tok"].long()
    ln_p = (z - s["norm"][:, :1]) / c["T"] - s["norm"][:, 1:]
    p = ln_p.exp()
    g = -p * (s["g_logp"][:, None] + s["g_ent"][:, None] * torch.where(p > 0, ln_p + s["entropy"][:, None], 0.0))
    rows = torch.arange(c["N"], device=z.device)
    g[rows, tok] += s["g_logp"]
    return (g / c["T"]).to(s["z"].dtype)


def _plain_embed(s):
    tok = s["tok"].long()
    rows = s["W"][tok.clamp(min=0)].float() * s["case"]["scale"]
    return torch.where(tok[:, None] >= 0, rows, 0.0).to(s["W"].dtype)


def _plain_embed_grad(s):
    c = s["case"]
    tok = s["tok"].long()
    g = torch.where(tok[:, None] >= 0, s["g"].float() * c["scale"], 0.0)
    out = torch.zeros(c["V"], c["D"], device=g.device)
    return out.index_add_(0, tok.clamp(min=0), g)


def _plain_bias_grad(s):
    G, a, W2 = s["G"].float(), s["a"].float(), s["W2"].float()
    if s["case"]["layout"] == "vr":
        return dict(grad_a=G @ W2, grad_W2=G.t() @ a)
    return dict(grad_a=G @ W2.t(), grad_W2=a.t() @ G)


_PLAIN = dict(logprob=_plain_logprob, logprob_grad=_plain_logprob_grad, embed=_plain_embed,
              embed_grad=_plain_embed_grad, bias_grad=_plain_bias_grad)


# ------------------------------------------------------------------ work
def work(case):
    k, N, V = case["kind"], case["N"], case["V"]
    es = 4 if case["dtype"] == "f32" else 2
    if k == "logprob":
        # logits and tokens in; log probability, two normalisers, entropy, rank, alternatives out.
        # Per entry: subtract, scale, exponential, two sums, one product, one comparison
        return {"bytes": N * V * es + N * 4 + N * 20 + N * case["top"] * 8, "flops": 7 * N * V}
    if k == "logprob_grad":
        return {"bytes": 2 * N * V * es + N * 24, "flops": 8 * N * V}
    if k == "embed":
        # a table row that several tokens share is read once
        rows = _expected_rows(N, V)
        return {"bytes": int((rows + N) * case["D"] * es) + N * 4, "flops": N * case["D"]}
    if k == "embed_grad":
        return {"bytes": N * case["D"] * es + N * 4 + V * case["D"] * 4, "flops": 2 * N * case["D"]}
    r, wes = case["r"], 4 if case["weights"] == "f32" else 2
    return {"bytes": N * V * es + (N + V) * r * wes + (N + V) * r * 4, "flops": 4 * N * V * r}


def _expected_rows(N, V):
    """Different tokens among N of the text distribution (rank's share ln((k + 2) / (k + 1)) / ln(V + 1))."""
    total, k = 0.0, 0
    while k < V:
        step = max(1, k // 64)
        share = math.log((k + 1.0 + step) / (k + 1.0)) / math.log(V + 1.0) / step
        total += min(step, V - k) * -math.expm1(N * math.log1p(-min(share, 1.0 - 1e-12)))
        k += step
    return total


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    x = _inputs(case, seed)
    k, N, V = case["kind"], case["N"], case["V"]
    if k == "logprob":
        T, parts = case["T"], []
        step = max(1, (1 << 25) // V)
        for i in range(0, N, step):
            z = x["z"][i:i + step].double()
            t = x["tok"][i:i + step].long()
            lse = torch.logsumexp(z / T, dim=1, keepdim=True)
            lp = z / T - lse
            p = lp.exp()
            zx = torch.take_along_dim(z, t[:, None], dim=1)
            m = z.amax(dim=1, keepdim=True)
            one = dict(logp=torch.take_along_dim(lp, t[:, None], dim=1)[:, 0],
                       norm=torch.cat([m, lse - m / T], dim=1),
                       entropy=torch.special.entr(p).sum(dim=1),
                       rank=(torch.count_nonzero(z > zx, dim=1) + 1).to(torch.int32))
            if case["top"]:
                _, ids = torch.sort(z, dim=1, descending=True, stable=True)
                ids = ids[:, :case["top"]]
                one.update(top_ids=ids.to(torch.int32), top_logp=torch.take_along_dim(lp, ids, dim=1))
            parts.append(one)
        return {n: torch.cat([q[n] for q in parts]) for n in parts[0]}
    if k == "logprob_grad":
        T, parts = case["T"], []
        step = max(1, (1 << 25) // V)
        for i in range(0, N, step):
            z = x["z"][i:i + step].double() / T
            t = x["tok"][i:i + step].long()
            p = torch.softmax(z, dim=1)
            lp = torch.log_softmax(z, dim=1)
            h = torch.special.entr(p).sum(dim=1, keepdim=True)
            gl, ge = x["g_logp"][i:i + step, None].double(), x["g_ent"][i:i + step, None].double()
            hot = torch.zeros_like(p).scatter_(1, t[:, None], 1.0)
            # kept in 32 bits: the largest of these results in 64 would not be worth its memory
            parts.append(((gl * (hot - p) - ge * (p * h - torch.special.entr(p))) / T).float()
                         if N * V > (1 << 28) else (gl * (hot - p) - ge * (p * h + p * lp)) / T)
        return torch.cat(parts)
    if k == "embed":
        table = torch.cat([x["W"], torch.zeros_like(x["W"][:1])])
        tok = x["tok"].long()
        return torch.index_select(table, 0, torch.where(tok < 0, V, tok)).double() * case["scale"]
    if k == "embed_grad":
        tok = x["tok"].long()
        keep = tok >= 0
        tok, g = tok[keep], x["g"][keep]
        order = torch.argsort(tok, stable=True)
        ids, counts = torch.unique_consecutive(tok[order], return_counts=True)
        out = torch.zeros(V, case["D"], dtype=torch.float64, device="cuda")
        if ids.numel():
            end = torch.cumsum(counts, 0)
            sums = torch.cumsum(g[order].double(), 0)[end - 1]
            sums[1:] -= sums[:-1].clone()
            out[ids] = sums * case["scale"]
        return out
    G, a, W2 = x["G"], x["a"].double(), x["W2"].double()
    if case["layout"] == "rv":
        W2 = W2.t()
    ga = torch.zeros(N, case["r"], dtype=torch.float64, device="cuda")
    gw = torch.empty(V, case["r"], dtype=torch.float64, device="cuda")
    step = max(1, (1 << 28) // max(N, 1))
    for v in range(0, V, step):
        part = G[:, v:v + step].double()
        ga += torch.mm(part, W2[v:v + step])
        gw[v:v + step] = torch.mm(part.t(), a)
    return dict(grad_a=ga, grad_W2=gw if case["layout"] == "vr" else gw.t().contiguous())
