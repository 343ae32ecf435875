"""libdspark Python binding: DSpark's semi-autoregressive draft-sampling hot path on GB300.

Every function here only marshals arguments: it checks dtypes and devices, allocates the
output tensors with PyTorch (device memory is PyTorch's job) and calls the C ABI declared in
``include/dspark.h``.  All arithmetic runs in the CUDA kernels of ``libdspark.so``; there is no
fallback path, and a missing library raises.

Names follow the pages: B requests, block size gamma, vocab V, Markov rank r, hidden size d,
temperature T; W1 (embedding, [V][r]), W2 (logit projection: [r][V] as the pages write it with
``w2_layout="rv"``, or a linear layer's [V][r] weight with the default ``"vr"``), w (confidence
weight [d + r]), Wj (RNN joint projection [3r][2r + d]), U (base logits [B][gamma][V]),
h (hidden states [B][gamma][d]), x0 (anchors [B]).

Beside the draft block: ``token_logprobs`` scores given tokens (log probability, entropy, rank,
alternatives), ``embedding`` looks rows of a table up, and ``token_logprobs_grad``, ``bias_grad`` and
``embedding_grad`` are the gradients that lead from a likelihood back to W1 and W2
(``examples/train_markov_head.py`` runs them together).  ``process_logits`` applies a request's penalties,
biases and grammar mask to its logits, before ``verify`` or any of these, and ``process_logits_grad`` leads
back through it; ``distill_loss`` and ``distill_grad`` train on a teacher's K largest log probabilities, which
``token_logprobs`` gives, where ``draft_loss`` takes whole target rows.  Each has a ``...Plan`` that checks and
marshals its arguments once.
"""
from __future__ import annotations

from contextlib import nullcontext
from dataclasses import dataclass

import torch

from . import _lib

__all__ = ["Workspace", "markov_draft", "rnn_draft", "confidence", "tv_label",
           "prefix_schedule", "draft_path", "draft_launches", "draft_loss_launches",
           "DraftOutput", "DraftPlan",
           "VerifyWorkspace", "verify", "LossWorkspace", "draft_loss", "sts", "CapacityRing",
           "LogprobWorkspace", "LogprobOutput", "LogprobPlan", "token_logprobs",
           "LogprobGradPlan", "token_logprobs_grad", "EmbeddingPlan", "embedding",
           "EmbeddingGradWorkspace", "EmbeddingGradPlan", "embedding_grad",
           "BiasGradWorkspace", "BiasGradPlan", "bias_grad",
           "ProcessPlan", "process_logits", "ProcessGradPlan", "process_logits_grad",
           "DistillWorkspace", "DistillOutput", "DistillPlan", "distill_loss", "DistillGradPlan", "distill_grad"]

_F32, _BF16 = 0, 1
_W2_LAYOUT = {"vr": 0, "rv": 1}


def _w2_code(layout: str) -> int:
    if layout not in _W2_LAYOUT:
        raise ValueError(f"w2_layout must be 'vr' ([V][r]) or 'rv' ([r][V]), not {layout!r}")
    return _W2_LAYOUT[layout]


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return _F32
    if t.dtype == torch.bfloat16:
        return _BF16
    raise TypeError(f"unsupported dtype {t.dtype}: use float32 or bfloat16")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libdspark takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libdspark takes contiguous tensors")
    return t.data_ptr()


def _stream(stream, device=None) -> int | None:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


class Workspace:
    """Zero-initialised device scratch for the draft calls; reusable across calls of the same
    or smaller shape, one call at a time (stream order)."""

    def __init__(self, head: int, B: int, gamma: int, V: int, r: int, d: int, device=None,
                 target: bool = False, w2_layout: str = "vr"):
        lib = _lib.load()
        flags = (1 if target else 0) | (2 if _w2_code(w2_layout) == 1 else 0)
        n = lib.dspark_workspace_bytes(head, B, gamma, V, r, d, flags)
        if n == 0:
            raise ValueError("invalid draft shape for a workspace")
        self.nbytes = int(n)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or "cuda")

    def status(self, stream=None) -> int:
        """Synchronise and read (then clear) the device status word."""
        return _lib.load().dspark_get_status(self.buf.data_ptr(), self.nbytes, _stream(stream))


@dataclass
class DraftOutput:
    tokens: torch.Tensor          # [B, gamma] int32
    lse: torch.Tensor             # [B, gamma] fp32, log-sum-exp of (U + B_k) / T
    c: torch.Tensor | None        # [B, gamma] Eq 7 confidence
    S: torch.Tensor | None        # [B, gamma] prefix survival
    cstar: torch.Tensor | None    # [B, gamma] Eq 8 soft acceptance label
    l1: torch.Tensor | None       # [B, gamma] ||p^d - p^t||_1
    logits: torch.Tensor | None   # [B, gamma, V] z = U + B_k (debug)
    s_out: torch.Tensor | None    # [B, r] final RNN state


class DraftPlan:
    """A draft call with its arguments marshalled once: ``run()`` enqueues it again with the
    same input and output buffers (one C call, no per-call allocation or checks)."""

    def __init__(self, head, W1, W2, U, x0, *, T, seed, h, w, Wj, target, forced, s0,
                 want_logits, workspace, stream, out=None, w2_layout="vr"):
        lib = _lib.load()
        B, gamma, V = U.shape
        r = W1.shape[1]
        d = h.shape[2] if h is not None else 0
        dev = U.device
        w2c = _w2_code(w2_layout)
        if tuple(W2.shape) != ((r, V) if w2c == 1 else (V, r)):
            raise ValueError(f"W2 must be {'[r][V]' if w2c == 1 else '[V][r]'} for w2_layout={w2_layout!r}")
        if workspace is None:
            workspace = Workspace(head, B, gamma, V, r, d, device=dev, target=target is not None,
                                  w2_layout=w2_layout)
        f32 = dict(dtype=torch.float32, device=dev)
        o = dict(out or {})
        conf = h is not None and w is not None

        def buf(name, shape, want, dtype=torch.float32):
            if not want:
                return None
            t = o.get(name)
            return t if t is not None else torch.empty(*shape, dtype=dtype, device=dev)

        tokens = buf("tokens", (B, gamma), True, torch.int32)
        lse = buf("lse", (B, gamma), True)
        c = buf("c", (B, gamma), conf)
        S = buf("S", (B, gamma), conf)
        cstar = buf("cstar", (B, gamma), target is not None)
        l1 = buf("l1", (B, gamma), target is not None)
        logits = buf("logits", (B, gamma, V), want_logits)
        s_out = buf("s_out", (B, r), head == 1)
        if x0.dtype != torch.int32 or (forced is not None and forced.dtype != torch.int32):
            raise TypeError("x0 and forced are int32")
        if target is not None and target.dtype != torch.float32:
            raise TypeError("target is float32")
        wdt, udt = _dtype_code(W1), _dtype_code(U)
        for t in (W2, w, Wj):
            if t is not None and _dtype_code(t) != wdt:
                raise TypeError("W1, W2, w and Wj share one dtype")
        if h is not None and _dtype_code(h) != udt:
            raise TypeError("U and h share one dtype")
        common_in = [_ptr(x0), _ptr(forced), _ptr(target)]
        outs = [_ptr(tokens), _ptr(lse), _ptr(c), _ptr(S), _ptr(cstar), _ptr(l1), _ptr(logits)]
        ws = [workspace.buf.data_ptr(), workspace.nbytes, _stream(stream)]
        if head == 0:
            self._fn = lib.dspark_markov_draft
            self._args = (B, gamma, V, r, d, float(T), int(seed), wdt, _ptr(W1), _ptr(W2), w2c,
                          _ptr(w), udt, _ptr(U), _ptr(h), *common_in, *outs, *ws)
            self._where = "dspark_markov_draft"
        else:
            self._fn = lib.dspark_rnn_draft
            self._args = (B, gamma, V, r, d, float(T), int(seed), wdt, _ptr(W1), _ptr(W2), w2c,
                          _ptr(w), _ptr(Wj), udt, _ptr(U), _ptr(h), *common_in, _ptr(s0), *outs,
                          _ptr(s_out), *ws)
            self._where = "dspark_rnn_draft"
        # keep every tensor whose address is baked into the arguments alive
        self._keep = (W1, W2, U, x0, h, w, Wj, target, forced, s0)
        self.workspace = workspace
        self.out = DraftOutput(tokens, lse, c, S, cstar, l1, logits, s_out)

    def run(self, stream=None) -> DraftOutput:
        """Enqueue the call; ``stream`` (a torch stream) overrides the one given at
        construction, e.g. the capturing stream of a CUDA graph."""
        args = self._args if stream is None else self._args[:-1] + (_stream(stream),)
        code = self._fn(*args)
        if code != 0:
            _lib.check(code, self._where)
        return self.out


def _draft(head, W1, W2, U, x0, **kw):
    return DraftPlan(head, W1, W2, U, x0, **kw).run()


def markov_draft(W1, W2, U, x0, *, T=1.0, seed=0, h=None, w=None, target=None, forced=None,
                 want_logits=False, workspace=None, stream=None, out=None,
                 w2_layout="vr") -> DraftOutput:
    """One draft block with the Markov head (Eq 5), sampling, Eq 7 confidence and S_k, and
    the Eq 8 label when ``target`` is given.  ``w2_layout``: "vr" for W2 [V][r], "rv" for
    [r][V].  See ``dspark_markov_draft``."""
    return _draft(0, W1, W2, U, x0, T=T, seed=seed, h=h, w=w, Wj=None, target=target,
                  forced=forced, s0=None, want_logits=want_logits, workspace=workspace,
                  stream=stream, out=out, w2_layout=w2_layout)


def rnn_draft(W1, W2, Wj, U, h, x0, *, T=1.0, seed=0, w=None, target=None, forced=None, s0=None,
              want_logits=False, workspace=None, stream=None, out=None,
              w2_layout="vr") -> DraftOutput:
    """One draft block with the RNN head (Eq 6).  See ``dspark_rnn_draft``."""
    return _draft(1, W1, W2, U, x0, T=T, seed=seed, h=h, w=w, Wj=Wj, target=target,
                  forced=forced, s0=s0, want_logits=want_logits, workspace=workspace,
                  stream=stream, out=out, w2_layout=w2_layout)


def confidence(W1, w, h, x0, tokens, *, stream=None):
    """Teacher-forced Eq 7 confidence and prefix survival for given tokens."""
    lib = _lib.load()
    B, gamma, d = h.shape
    V, r = W1.shape
    c = torch.empty(B, gamma, dtype=torch.float32, device=h.device)
    S = torch.empty_like(c)
    code = lib.dspark_confidence(B, gamma, V, r, d, _dtype_code(W1), _ptr(W1), _ptr(w),
                                 _dtype_code(h), _ptr(h), _ptr(x0), _ptr(tokens), _ptr(c),
                                 _ptr(S), _stream(stream))
    _lib.check(code, "dspark_confidence")
    return c, S


def tv_label(draft_logits, target_logits, *, T=1.0, stream=None):
    """Eq 8 soft acceptance label c* and the L1 distance on [N, V] fp32 logit rows."""
    lib = _lib.load()
    N, V = draft_logits.shape
    cstar = torch.empty(N, dtype=torch.float32, device=draft_logits.device)
    l1 = torch.empty_like(cstar)
    code = lib.dspark_tv_label(N, V, float(T), _ptr(draft_logits), _ptr(target_logits),
                               _ptr(cstar), _ptr(l1), _stream(stream))
    _lib.check(code, "dspark_tv_label")
    return cstar, l1


def prefix_schedule(S, sps, *, stream=None, out=None):
    """Per-request verify lengths maximising SPS(n) * expected accepted tokens.

    ``out``: optional preallocated (lengths [B] int32, theta [1] float64) device tensors, e.g.
    to capture the call in a CUDA graph."""
    lib = _lib.load()
    B, gamma = S.shape
    if out is not None:
        ln, theta = out
    else:
        ln = torch.empty(B, dtype=torch.int32, device=S.device)
        theta = torch.empty(1, dtype=torch.float64, device=S.device)
    code = lib.dspark_prefix_schedule(B, gamma, _ptr(S), _ptr(sps), _ptr(ln), _ptr(theta),
                                      _stream(stream))
    _lib.check(code, "dspark_prefix_schedule")
    return ln, theta


class VerifyWorkspace(Workspace):
    """Zero-initialised device scratch for ``verify`` (shapes up to B, gamma, V)."""

    def __init__(self, B: int, gamma: int, V: int, device=None):
        n = _lib.load().dspark_verify_workspace_bytes(B, gamma, V)
        if n == 0:
            raise ValueError("invalid verify shape for a workspace")
        self.nbytes = int(n)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or "cuda")


def verify(draft_logits, target_logits, draft_tokens, *, T=1.0, seed=0, workspace=None,
           stream=None, out=None):
    """Speculative accept/reject of one draft block per request.  See ``dspark_verify``.

    draft_logits [B, gamma, V] fp32, target_logits [B, gamma + 1, V] fp32, draft_tokens
    [B, gamma] int32.  Returns (n_accepted [B] int32, out_tokens [B, gamma + 1] int32).
    """
    lib = _lib.load()
    B, gamma, V = draft_logits.shape
    if draft_logits.dtype != torch.float32 or target_logits.dtype != torch.float32:
        raise TypeError("verify takes fp32 logits")
    if tuple(target_logits.shape) != (B, gamma + 1, V) or tuple(draft_tokens.shape) != (B, gamma):
        raise ValueError("target_logits must be [B, gamma + 1, V] and draft_tokens [B, gamma]")
    ws = workspace or VerifyWorkspace(B, gamma, V, device=draft_logits.device)
    if out is None:
        n = torch.empty(B, dtype=torch.int32, device=draft_logits.device)
        toks = torch.empty(B, gamma + 1, dtype=torch.int32, device=draft_logits.device)
    else:
        n, toks = out
    code = lib.dspark_verify(B, gamma, V, float(T), int(seed) & (2**64 - 1), _ptr(draft_logits),
                             _ptr(target_logits), _ptr(draft_tokens), _ptr(n), _ptr(toks),
                             ws.buf.data_ptr(), ws.nbytes, _stream(stream))
    _lib.check(code, "dspark_verify")
    return n, toks


class LossWorkspace(Workspace):
    """Device scratch for ``draft_loss`` (shapes up to B, gamma, V)."""

    def __init__(self, B: int, gamma: int, V: int, device=None):
        n = _lib.load().dspark_draft_loss_workspace_bytes(B, gamma, V)
        if n == 0:
            raise ValueError("invalid loss shape for a workspace")
        self.nbytes = int(n)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or "cuda")


def draft_loss(draft_logits, target_logits, labels, conf_logits, *, T=1.0,
               alpha=(0.1, 0.9, 1.0), want_grads=True, workspace=None, stream=None):
    """Eqs 9-12 and their gradients (c* held as a label).  See ``dspark_draft_loss``.

    Returns (loss [B], parts [B, 3], grad_logits [B, gamma, V] or None, grad_conf [B, gamma]
    or None), all fp32.
    """
    lib = _lib.load()
    B, gamma, V = draft_logits.shape
    if draft_logits.dtype != torch.float32 or target_logits.dtype != torch.float32:
        raise TypeError("draft_loss takes fp32 logits")
    dev = draft_logits.device
    ws = workspace or LossWorkspace(B, gamma, V, device=dev)
    loss = torch.empty(B, dtype=torch.float32, device=dev)
    parts = torch.empty(B, 3, dtype=torch.float32, device=dev)
    gz = torch.empty_like(draft_logits) if want_grads else None
    gc = torch.empty(B, gamma, dtype=torch.float32, device=dev) if want_grads else None
    code = lib.dspark_draft_loss(B, gamma, V, float(T), _ptr(draft_logits), _ptr(target_logits),
                                 _ptr(labels), _ptr(conf_logits), float(alpha[0]),
                                 float(alpha[1]), float(alpha[2]), _ptr(loss), _ptr(parts),
                                 _ptr(gz), _ptr(gc), ws.buf.data_ptr(), ws.nbytes, _stream(stream))
    _lib.check(code, "dspark_draft_loss")
    return loss, parts, gz, gc


def sts(conf_logits, accepted, grid, *, bins=15, stream=None):
    """Sequential temperature scaling of the confidence head.  See ``dspark_sts``.

    conf_logits [N, gamma] fp32, accepted [N] int32, grid [ngrid] fp32.  Returns (tau [gamma],
    ece [gamma], ece_grid [gamma, ngrid]) fp32 and the device status.
    """
    lib = _lib.load()
    N, gamma = conf_logits.shape
    ng = grid.shape[0]
    n = lib.dspark_sts_workspace_bytes(N, gamma, ng, bins)
    if n == 0:
        raise ValueError("invalid sts shape")
    ws = Workspace.__new__(Workspace)
    ws.nbytes = int(n)
    ws.buf = torch.zeros(ws.nbytes, dtype=torch.uint8, device=conf_logits.device)
    tau = torch.empty(gamma, dtype=torch.float32, device=conf_logits.device)
    ece = torch.empty_like(tau)
    eg = torch.empty(gamma, ng, dtype=torch.float32, device=conf_logits.device)
    code = lib.dspark_sts(N, gamma, _ptr(conf_logits), _ptr(accepted), ng, _ptr(grid), bins,
                          _ptr(tau), _ptr(ece), _ptr(eg), ws.buf.data_ptr(), ws.nbytes,
                          _stream(stream))
    _lib.check(code, "dspark_sts")
    return tau, ece, eg, ws.status(stream)


class _Plan:
    """A call with its arguments checked and marshalled once: ``run()`` enqueues it again with the
    same input and output buffers (one C call, no per-call allocation or checks) and returns
    ``out``.  ``stream`` (a torch stream) overrides the one given at construction.

    What a plan allocates (outputs, workspace) belongs to its stream: given ``stream``, it is
    allocated and cleared there.  Everything that the call reads or writes, a caller's outputs and
    workspace among it, is recorded as in use on a stream that was given.  The first run on a stream other
    than the plan's waits for what the plan's has enqueued so far (the clearing of the workspace); later
    ones are ordered by the caller, and so is a run that a graph captures."""

    def _set(self, name, args, stream, out, keep, device):
        self._fn = getattr(_lib.load(), name)
        self._where = name
        self._index = device.index
        self._stream = stream if stream is not None else torch.cuda.current_stream(device)
        self._args = (*args, self._stream.cuda_stream)
        self._others = {}   # streams of other runs, by handle
        self.out = out
        self._keep = (keep, out)   # everything whose address is baked into the arguments stays alive
        if stream is not None:
            self._record(stream)

    def _record(self, stream):
        for t in _tensors(self._keep):
            t.record_stream(stream)

    def _elsewhere(self, stream):
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return
        stream.wait_stream(self._stream)
        self._record(stream)
        self._others[stream.cuda_stream] = stream

    def run(self, stream=None):
        _check_current(self._index)
        args = self._args
        if stream is not None and stream.cuda_stream != args[-1]:
            if stream.cuda_stream not in self._others:
                self._elsewhere(stream)
            args = args[:-1] + (stream.cuda_stream,)
        code = self._fn(*args)
        if code != 0:
            _lib.check(code, self._where)
        return self.out


def _tensors(items):
    """The tensors of nested tuples, workspaces and outputs."""
    for x in items:
        if isinstance(x, torch.Tensor):
            yield x
        elif isinstance(x, Workspace):
            yield x.buf
        elif isinstance(x, tuple):
            yield from _tensors(x)
        elif isinstance(x, (LogprobOutput, DistillOutput)):
            yield from _tensors(vars(x).values())


def _on(stream):
    """The context in which a plan's own tensors are allocated."""
    return torch.cuda.stream(stream) if stream is not None else nullcontext()


def _same_device(*tensors):
    """The device of all these tensors (and workspaces), which is the current one: the library
    launches there."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if isinstance(t, Workspace):
            t = t.buf
        if not t.is_cuda:
            raise ValueError("libdspark takes device tensors")
        if dev is not None and t.device != dev:
            raise ValueError("all tensors are on one device")
        dev = t.device
    _check_current(dev.index)
    return dev


def _check_current(index):
    if torch.cuda.current_device() != index:
        raise ValueError(f"the tensors are on cuda:{index}, which is not the current device")


def _ints(t, shape, name):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != torch.int32:
        raise TypeError(f"{name} is int32")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    return _ptr(t)


def _f32(t, shape, name):
    if t is None:
        return None
    if t.dtype != torch.float32:
        raise TypeError(f"{name} is float32")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    return _ptr(t)


def _logit_rows(z, name):
    """(leading shape, N, V, row stride, address) of logits [..., V]: the entries of a row are
    consecutive, and the rows are one stride apart (a slice of a padded vocabulary is fine)."""
    if z.dim() < 1 or z.shape[-1] < 2:
        raise ValueError(f"{name} must be [..., V] with V >= 2")
    if not z.is_cuda:
        raise ValueError("libdspark takes device tensors")
    lead, V = tuple(z.shape[:-1]), z.shape[-1]
    N = 1
    for n in lead:
        N *= n
    if N == 0:
        return lead, 0, V, V, None
    if z.stride(-1) != 1:
        raise ValueError(f"the entries of a row of {name} are consecutive in memory")
    ld = None   # the stride of the flattened leading dimensions
    inner = 1
    for n, st in zip(reversed(lead), reversed(z.stride()[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld = st
        elif st != ld * inner:
            raise ValueError(f"the rows of {name} are not one stride apart: make it contiguous")
        inner *= n
    ld = V if ld is None else ld
    if ld < V:
        raise ValueError(f"the rows of {name} overlap")
    return lead, N, V, ld, z.data_ptr()


class LogprobWorkspace(Workspace):
    """Zero-initialised device scratch for ``token_logprobs`` (shapes up to N rows, V, top)."""

    def __init__(self, N: int, V: int, top: int = 0, device=None):
        n = _lib.load().dspark_token_logprobs_workspace_bytes(N, V, top)
        if n == 0:
            raise ValueError("invalid token_logprobs shape for a workspace")
        self.nbytes = int(n)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or "cuda")


@dataclass
class LogprobOutput:
    logp: torch.Tensor            # [...] ln p of the given token
    norm: torch.Tensor            # [..., 2] (largest logit, ln sum exp((z - largest) / T))
    entropy: torch.Tensor         # [...]
    rank: torch.Tensor            # [...] int32, 1 for the largest logit
    top_ids: torch.Tensor | None  # [..., top] int32, -1 past the last alternative
    top_logp: torch.Tensor | None  # [..., top]


class LogprobPlan(_Plan):
    """``token_logprobs`` with its arguments marshalled once (see ``_Plan``)."""

    def __init__(self, logits, tokens, *, T=1.0, top=0, workspace=None, stream=None, out=None):
        dev = _same_device(logits, tokens, workspace)
        zdt = _dtype_code(logits)
        lead, N, V, ld, zp = _logit_rows(logits, "logits")
        if not 0 <= top <= min(32, V):
            raise ValueError("top must be 0..min(32, V)")
        tp = _ints(tokens, lead, "tokens")
        with _on(stream):
            ws = workspace or LogprobWorkspace(N, V, top, device=dev)
            if out is None:
                def new(*shape, dtype=torch.float32):
                    return torch.empty((*lead, *shape), dtype=dtype, device=dev)
                out = LogprobOutput(new(), new(2), new(), new(dtype=torch.int32),
                                    new(top, dtype=torch.int32) if top else None, new(top) if top else None)
        _same_device(logits, out.logp, out.norm, out.entropy, out.rank, out.top_ids, out.top_logp)
        args = (N, V, float(T), zdt, zp, ld, tp, top, _f32(out.logp, lead, "logp"),
                _f32(out.norm, (*lead, 2), "norm"), _f32(out.entropy, lead, "entropy"),
                _ints(out.rank, lead, "rank"),
                _ints(out.top_ids, (*lead, top), "top_ids") if top else None,
                _f32(out.top_logp, (*lead, top), "top_logp") if top else None, ws.buf.data_ptr(), ws.nbytes)
        self.workspace = ws
        self._set("dspark_token_logprobs", args, stream, out, (logits, tokens, ws), dev)


def token_logprobs(logits, tokens, *, T=1.0, top=0, workspace=None, stream=None,
                   out=None) -> LogprobOutput:
    """Log probabilities of given tokens under softmax(logits / T), with the entropy, the tokens'
    ranks and the ``top`` (<= 32) most likely alternatives.  See ``dspark_token_logprobs``.

    logits [..., V] fp32 or bf16 (rows one stride apart), tokens [...] int32, -1 for no token.
    ``out``: an earlier call's LogprobOutput to write into."""
    return LogprobPlan(logits, tokens, T=T, top=top, workspace=workspace, stream=stream, out=out).run()


class LogprobGradPlan(_Plan):
    """``token_logprobs_grad`` with its arguments marshalled once (see ``_Plan``)."""

    def __init__(self, logits, tokens, norm, *, T=1.0, grad_logp=None, grad_entropy=None, entropy=None,
                 stream=None, out=None):
        dev = _same_device(logits, tokens, norm, entropy, grad_logp, grad_entropy, out)
        if out is None:
            with _on(stream):
                out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        zdt = _dtype_code(logits)
        lead, N, V, ld, zp = _logit_rows(logits, "logits")
        if out.dtype != logits.dtype or out.shape != logits.shape:
            raise ValueError("out has the logits' shape and dtype")
        if grad_logp is None and grad_entropy is None:
            raise ValueError("grad_logp or grad_entropy is required")
        if grad_entropy is not None and entropy is None:
            raise ValueError("grad_entropy needs the forward call's entropy")
        _, _, _, gld, gp = _logit_rows(out, "out")
        args = (N, V, float(T), zdt, zp, ld, _ints(tokens, lead, "tokens"), _f32(norm, (*lead, 2), "norm"),
                _f32(entropy, lead, "entropy"), _f32(grad_logp, lead, "grad_logp"),
                _f32(grad_entropy, lead, "grad_entropy"), gp, gld)
        self._set("dspark_token_logprobs_grad", args, stream, out,
                  (logits, tokens, norm, entropy, grad_logp, grad_entropy), dev)


def token_logprobs_grad(logits, tokens, norm, *, T=1.0, grad_logp=None, grad_entropy=None,
                        entropy=None, stream=None, out=None):
    """Gradient of ``token_logprobs``' logp and entropy with respect to the logits, in their dtype.

    ``norm`` and ``entropy`` are the forward call's; grad_logp, grad_entropy [...] fp32 (at least
    one).  ``out`` may be the logits themselves.  See ``dspark_token_logprobs_grad``."""
    return LogprobGradPlan(logits, tokens, norm, T=T, grad_logp=grad_logp, grad_entropy=grad_entropy,
                           entropy=entropy, stream=stream, out=out).run()


class EmbeddingPlan(_Plan):
    """``embedding`` with its arguments marshalled once (see ``_Plan``)."""

    def __init__(self, W, tokens, *, scale=1.0, dtype=None, stream=None, out=None):
        dev = _same_device(W, tokens, out)
        V, D = W.shape
        lead = tuple(tokens.shape)
        if out is None:
            with _on(stream):
                out = torch.empty(*lead, D, dtype=dtype or W.dtype, device=dev)
        elif tuple(out.shape) != (*lead, D) or (dtype is not None and out.dtype != dtype):
            raise ValueError("out must be [..., D] of the requested dtype")
        args = (tokens.numel(), V, D, float(scale), _dtype_code(W), _ptr(W), _ints(tokens, lead, "tokens"),
                _dtype_code(out), _ptr(out))
        self._set("dspark_embedding", args, stream, out, (W, tokens), dev)


def embedding(W, tokens, *, scale=1.0, dtype=None, stream=None, out=None):
    """scale * W[tokens]: rows of W [V, D] for tokens [...] int32, zero rows for -1, in ``dtype``
    (W's by default).  See ``dspark_embedding``."""
    return EmbeddingPlan(W, tokens, scale=scale, dtype=dtype, stream=stream, out=out).run()


class EmbeddingGradWorkspace(Workspace):
    """Zero-initialised device scratch for ``embedding_grad`` (shapes up to N tokens, V, D)."""

    def __init__(self, N: int, V: int, D: int, device=None):
        n = _lib.load().dspark_embedding_grad_workspace_bytes(N, V, D)
        if n == 0:
            raise ValueError("invalid embedding_grad shape for a workspace")
        self.nbytes = int(n)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or "cuda")


class EmbeddingGradPlan(_Plan):
    """``embedding_grad`` with its arguments marshalled once (see ``_Plan``)."""

    def __init__(self, grad, tokens, V, *, scale=1.0, dtype=torch.float32, accumulate=False, out=None,
                 workspace=None, stream=None):
        dev = _same_device(grad, tokens, out, workspace)
        lead, D = tuple(tokens.shape), grad.shape[-1]
        if tuple(grad.shape) != (*lead, D):
            raise ValueError("grad must be [..., D] for tokens [...]")
        N = tokens.numel()
        if out is None:
            if accumulate:
                raise ValueError("accumulate adds to out: give it")
            with _on(stream):
                out = torch.empty(V, D, dtype=dtype, device=dev)
        elif tuple(out.shape) != (V, D):
            raise ValueError("out must be [V, D]")
        with _on(stream):
            ws = workspace or EmbeddingGradWorkspace(N, V, D, device=dev)
        args = (N, V, D, float(scale), _dtype_code(grad), _ptr(grad), _ints(tokens, lead, "tokens"),
                _dtype_code(out), _ptr(out), int(accumulate), ws.buf.data_ptr(), ws.nbytes)
        self.workspace = ws
        self._set("dspark_embedding_grad", args, stream, out, (grad, tokens, ws), dev)


def embedding_grad(grad, tokens, V, *, scale=1.0, dtype=torch.float32, accumulate=False, out=None,
                   workspace=None, stream=None):
    """The table gradient [V, D] of ``embedding``: every token's rows of grad [..., D] summed and
    scaled; ``accumulate`` adds them to ``out``.  See ``dspark_embedding_grad``."""
    return EmbeddingGradPlan(grad, tokens, V, scale=scale, dtype=dtype, accumulate=accumulate, out=out,
                             workspace=workspace, stream=stream).run()


class BiasGradWorkspace(Workspace):
    """Zero-initialised device scratch for ``bias_grad`` of this shape (or fewer rows)."""

    def __init__(self, N: int, V: int, r: int, bf16: bool = True, device=None):
        n = _lib.load().dspark_bias_grad_workspace_bytes(N, V, r, _BF16 if bf16 else _F32)
        if n == 0:
            raise ValueError("invalid bias_grad shape for a workspace")
        self.nbytes = int(n)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or "cuda")


class BiasGradPlan(_Plan):
    """``bias_grad`` with its arguments marshalled once (see ``_Plan``)."""

    def __init__(self, grad_logits, a, W2, *, w2_layout="vr", accumulate=False, out=None, workspace=None,
                 stream=None):
        dev = _same_device(grad_logits, a, W2, workspace)
        V, r = grad_logits.shape[-1], a.shape[-1]
        lead = tuple(grad_logits.shape[:-1])
        w2c = _w2_code(w2_layout)
        if tuple(a.shape) != (*lead, r) or tuple(W2.shape) != ((r, V) if w2c == 1 else (V, r)):
            raise ValueError("a must be [..., r] for grad_logits [..., V], and W2 [V][r] or [r][V] by w2_layout")
        wdt = _dtype_code(a)
        if _dtype_code(W2) != wdt:
            raise TypeError("a and W2 share one dtype")
        N = 1
        for n in lead:
            N *= n
        if out is None:
            if accumulate:
                raise ValueError("accumulate adds to out: give it")
            with _on(stream):
                out = (torch.empty(*lead, r, dtype=torch.float32, device=dev),
                       torch.empty(W2.shape, dtype=torch.float32, device=dev))
        _same_device(grad_logits, *out)
        with _on(stream):
            ws = workspace or BiasGradWorkspace(N, V, r, wdt == _BF16, device=dev)
        args = (N, V, r, _dtype_code(grad_logits), _ptr(grad_logits), wdt, _ptr(a), _ptr(W2), w2c,
                _f32(out[0], (*lead, r), "grad_a"), _f32(out[1], W2.shape, "grad_W2"), int(accumulate),
                ws.buf.data_ptr(), ws.nbytes)
        self.workspace = ws
        self._set("dspark_bias_grad", args, stream, tuple(out), (grad_logits, a, W2, ws), dev)


def bias_grad(grad_logits, a, W2, *, w2_layout="vr", accumulate=False, out=None, workspace=None,
              stream=None):
    """Gradients of the bias product a W2 (Eqs 5, 6) for logit gradients [..., V]: (grad_a [..., r],
    grad_W2 in W2's layout), fp32; ``accumulate`` adds to ``out[1]``.  See ``dspark_bias_grad``."""
    return BiasGradPlan(grad_logits, a, W2, w2_layout=w2_layout, accumulate=accumulate, out=out,
                        workspace=workspace, stream=stream).run()


def _history(history, B):
    """(address, row stride, H) of histories [B, H]: the tokens of a row are consecutive."""
    if history is None:
        return None, 0, 0
    if history.dtype != torch.int32:
        raise TypeError("history is int32")
    if history.dim() != 2 or history.shape[0] != B:
        raise ValueError(f"history must be [{B}, H], not {list(history.shape)}")
    H = history.shape[1]
    if H == 0 or B == 0:
        return None, H, 0
    ld = history.stride(0) if B > 1 else H
    if (H > 1 and history.stride(1) != 1) or ld < H:
        raise ValueError("the tokens of a row of history are consecutive, and its rows do not overlap")
    return history.data_ptr(), ld, H


def _mask(mask, mask_rows, lead, V):
    """(address, row stride, rows, address of the rows' choice) of a mask [M, words] int32."""
    if mask is None:
        if mask_rows is not None:
            raise ValueError("mask_rows needs mask")
        return None, 0, 0, None
    if mask.dtype != torch.int32:
        raise TypeError("mask is int32: 32 entries a word")
    if mask.dim() != 2 or mask.shape[1] < (V + 31) // 32:
        raise ValueError(f"mask must be [M, >= {(V + 31) // 32}], not {list(mask.shape)}")
    M = mask.shape[0]
    ld = mask.stride(0) if M > 1 else mask.shape[1]
    if (mask.shape[1] > 1 and mask.stride(1) != 1) or ld < mask.shape[1]:
        raise ValueError("the words of a row of mask are consecutive, and its rows do not overlap")
    N = 1
    for n in lead:
        N *= n
    if mask_rows is None and M != N:
        raise ValueError(f"mask needs a row for each of {N} rows, or mask_rows")
    return mask.data_ptr(), ld, M, _ints(mask_rows, lead, "mask_rows") if mask_rows is not None else None


def _block(logits, name):
    """(leading shape, B, R, V, row stride, address) of logits [B, V] or [B, R, V]."""
    if logits.dim() not in (2, 3):
        raise ValueError(f"{name} must be [B, V] or [B, R, V]")
    lead, _, V, ld, p = _logit_rows(logits, name)
    return lead, lead[0], lead[1] if len(lead) == 2 else 1, V, ld, p


def _requests(B, R, lengths, prompt_lengths, drafted, history):
    if history is None and (lengths is not None or prompt_lengths is not None):
        raise ValueError("lengths and prompt_lengths need history")
    return (_ints(lengths, (B,), "lengths") if lengths is not None else None,
            _ints(prompt_lengths, (B,), "prompt_lengths") if prompt_lengths is not None else None,
            _ints(drafted, (B, R - 1), "drafted") if drafted is not None else None)


class ProcessPlan(_Plan):
    """``process_logits`` with its arguments marshalled once (see ``_Plan``)."""

    def __init__(self, logits, *, history=None, lengths=None, prompt_lengths=None, drafted=None, repetition=None,
                 presence=None, frequency=None, bias_tokens=None, bias=None, mask=None, mask_rows=None, dtype=None,
                 stream=None, out=None):
        keep = (logits, history, lengths, prompt_lengths, drafted, repetition, presence, frequency, bias_tokens,
                bias, mask, mask_rows)
        dev = _same_device(*keep, out)
        zdt = _dtype_code(logits)
        lead, B, R, V, ld, zp = _block(logits, "logits")
        if out is None:
            with _on(stream):
                out = torch.empty(logits.shape, dtype=dtype or logits.dtype, device=dev)
        elif out.shape != logits.shape or (dtype is not None and out.dtype != dtype):
            raise ValueError("out has the logits' shape, and the requested dtype")
        odt = _dtype_code(out)
        _, _, _, old, op = _logit_rows(out, "out")
        if (bias_tokens is None) != (bias is None):
            raise ValueError("bias_tokens and bias go together")
        nb = bias.shape[-1] if bias is not None else 0
        hp, hld, H = _history(history, B)
        mp, mld, M, rows = _mask(mask, mask_rows, lead, V)
        args = (B, R, V, zdt, zp, ld, hp, hld, H, *_requests(B, R, lengths, prompt_lengths, drafted, history),
                _f32(repetition, (B,), "repetition"), _f32(presence, (B,), "presence"),
                _f32(frequency, (B,), "frequency"), nb,
                _ints(bias_tokens, (B, nb), "bias_tokens") if nb else None, _f32(bias, (B, nb), "bias"),
                mp, mld, M, rows, odt, op, old)
        self._set("dspark_process_logits", args, stream, out, keep, dev)


def process_logits(logits, *, history=None, lengths=None, prompt_lengths=None, drafted=None, repetition=None,
                   presence=None, frequency=None, bias_tokens=None, bias=None, mask=None, mask_rows=None, dtype=None,
                   stream=None, out=None):
    """A request's penalties, biases and grammar mask applied to its logits, in ``dtype`` (the logits' by
    default).  See ``dspark_process_logits``.

    logits [B, V], or [B, R, V] for blocks, fp32 or bf16 (rows one stride apart); history [B, H] int32 with
    ``lengths`` and ``prompt_lengths`` [B] int32; drafted [B, R - 1] int32, which row k counts the first k of;
    repetition, presence, frequency [B] fp32; bias_tokens, bias [B, nb]; mask [M, >= ceil(V / 32)] int32 words of
    bits, a set bit allowing its entry, and mask_rows [B] or [B, R] int32 (-1: no mask).  ``out`` may be the
    logits themselves."""
    return ProcessPlan(logits, history=history, lengths=lengths, prompt_lengths=prompt_lengths, drafted=drafted,
                       repetition=repetition, presence=presence, frequency=frequency, bias_tokens=bias_tokens,
                       bias=bias, mask=mask, mask_rows=mask_rows, dtype=dtype, stream=stream, out=out).run()


class ProcessGradPlan(_Plan):
    """``process_logits_grad`` with its arguments marshalled once (see ``_Plan``)."""

    def __init__(self, grad, logits, *, history=None, lengths=None, prompt_lengths=None, drafted=None,
                 repetition=None, mask=None, mask_rows=None, stream=None, out=None):
        keep = (grad, logits, history, lengths, prompt_lengths, drafted, repetition, mask, mask_rows)
        dev = _same_device(*keep, out)
        gdt, zdt = _dtype_code(grad), _dtype_code(logits)
        lead, B, R, V, ld, zp = _block(logits, "logits")
        if grad.shape != logits.shape:
            raise ValueError("grad has the logits' shape")
        if out is None:
            with _on(stream):
                out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        elif out.shape != logits.shape or out.dtype != logits.dtype:
            raise ValueError("out has the logits' shape and dtype")
        _, _, _, gld, gp = _logit_rows(grad, "grad")
        _, _, _, old, op = _logit_rows(out, "out")
        hp, hld, H = _history(history, B)
        mp, mld, M, rows = _mask(mask, mask_rows, lead, V)
        args = (B, R, V, gdt, gp, gld, zdt, zp, ld, hp, hld, H,
                *_requests(B, R, lengths, prompt_lengths, drafted, history), _f32(repetition, (B,), "repetition"),
                mp, mld, M, rows, op, old)
        self._set("dspark_process_logits_grad", args, stream, out, keep, dev)


def process_logits_grad(grad, logits, *, history=None, lengths=None, prompt_lengths=None, drafted=None,
                        repetition=None, mask=None, mask_rows=None, stream=None, out=None):
    """Gradient with respect to the raw logits, in their dtype, for the gradient ``grad`` with respect to what
    ``process_logits`` made of them (fp32 or bf16).  ``out`` may be ``grad`` itself.  See
    ``dspark_process_logits_grad``."""
    return ProcessGradPlan(grad, logits, history=history, lengths=lengths, prompt_lengths=prompt_lengths,
                           drafted=drafted, repetition=repetition, mask=mask, mask_rows=mask_rows, stream=stream,
                           out=out).run()


class DistillWorkspace(Workspace):
    """Zero-initialised device scratch for ``distill_loss`` and ``distill_grad`` (shapes up to N rows, V, K)."""

    def __init__(self, N: int, V: int, K: int, device=None):
        n = _lib.load().dspark_distill_workspace_bytes(N, V, K)
        if n == 0:
            raise ValueError("invalid distillation shape for a workspace")
        self.nbytes = int(n)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or "cuda")


@dataclass
class DistillOutput:
    loss: torch.Tensor                # [...]
    parts: torch.Tensor               # [..., 2] (KL, L1), without their weights
    norm: torch.Tensor                # [..., 4] (largest logit, ln sum) of the row and outside the teacher's tokens
    grad_logits: torch.Tensor | None  # the logits' shape and dtype


def _teacher(teacher_ids, teacher_logp, lead):
    K = teacher_ids.shape[-1] if teacher_ids.dim() else 0
    return K, _ints(teacher_ids, (*lead, K), "teacher_ids"), _f32(teacher_logp, (*lead, K), "teacher_logp")


class DistillPlan(_Plan):
    """``distill_loss`` with its arguments marshalled once (see ``_Plan``)."""

    def __init__(self, logits, teacher_ids, teacher_logp, *, T=1.0, alpha=(1.0, 0.0), rest=True, weight=None,
                 want_grad=True, workspace=None, stream=None, out=None):
        dev = _same_device(logits, teacher_ids, teacher_logp, weight, workspace)
        zdt = _dtype_code(logits)
        lead, N, V, ld, zp = _logit_rows(logits, "logits")
        K, ip, lp = _teacher(teacher_ids, teacher_logp, lead)
        with _on(stream):
            ws = workspace or DistillWorkspace(N, V, K, device=dev)
            if out is None:
                def new(*shape):
                    return torch.empty((*lead, *shape), dtype=torch.float32, device=dev)
                grad = torch.empty(logits.shape, dtype=logits.dtype, device=dev) if want_grad else None
                out = DistillOutput(new(), new(2), new(4), grad)
        _same_device(logits, out.loss, out.parts, out.norm, out.grad_logits)
        gp, gld = None, V
        if want_grad:
            if out.grad_logits is None:
                raise ValueError("out has no grad_logits")
            if out.grad_logits.shape != logits.shape or out.grad_logits.dtype != logits.dtype:
                raise ValueError("grad_logits has the logits' shape and dtype")
            _, _, _, gld, gp = _logit_rows(out.grad_logits, "grad_logits")
        args = (N, V, float(T), zdt, zp, ld, K, ip, lp, _f32(weight, lead, "weight"), float(alpha[0]),
                float(alpha[1]), int(bool(rest)), _f32(out.loss, lead, "loss"), _f32(out.parts, (*lead, 2), "parts"),
                _f32(out.norm, (*lead, 4), "norm"), gp, gld, ws.buf.data_ptr(), ws.nbytes)
        self.workspace = ws
        self._set("dspark_distill_loss", args, stream, out, (logits, teacher_ids, teacher_logp, weight, ws), dev)


def distill_loss(logits, teacher_ids, teacher_logp, *, T=1.0, alpha=(1.0, 0.0), rest=True, weight=None,
                 want_grad=True, workspace=None, stream=None, out=None) -> DistillOutput:
    """Loss of softmax(logits / T) against a teacher's K (<= 128) largest log probabilities: ``alpha[0]`` times
    their relative entropy plus ``alpha[1]`` times their L1 distance, each over the K tokens and, with
    ``rest``, everything else as one more outcome; with its gradient in the same call (``want_grad``).  See
    ``dspark_distill_loss``.

    logits [..., V] fp32 or bf16 (rows one stride apart), teacher_ids [..., K] int32 (-1: none) and teacher_logp
    [..., K] fp32, as ``token_logprobs(..., top=K)`` gives them; weight [...] fp32 (0: a padding row).  ``out``: an
    earlier call's DistillOutput, whose grad_logits may be the logits themselves."""
    return DistillPlan(logits, teacher_ids, teacher_logp, T=T, alpha=alpha, rest=rest, weight=weight,
                       want_grad=want_grad, workspace=workspace, stream=stream, out=out).run()


class DistillGradPlan(_Plan):
    """``distill_grad`` with its arguments marshalled once (see ``_Plan``)."""

    def __init__(self, logits, teacher_ids, teacher_logp, norm, grad_loss, *, T=1.0, alpha=(1.0, 0.0), rest=True,
                 workspace=None, stream=None, out=None):
        dev = _same_device(logits, teacher_ids, teacher_logp, norm, grad_loss, workspace, out)
        zdt = _dtype_code(logits)
        lead, N, V, ld, zp = _logit_rows(logits, "logits")
        K, ip, lp = _teacher(teacher_ids, teacher_logp, lead)
        with _on(stream):
            ws = workspace or DistillWorkspace(N, V, K, device=dev)
            if out is None:
                out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        if out.shape != logits.shape or out.dtype != logits.dtype:
            raise ValueError("out has the logits' shape and dtype")
        if norm is None or grad_loss is None:
            raise ValueError("norm and grad_loss are required")
        _, _, _, gld, gp = _logit_rows(out, "out")
        args = (N, V, float(T), zdt, zp, ld, K, ip, lp, _f32(norm, (*lead, 4), "norm"),
                _f32(grad_loss, lead, "grad_loss"), float(alpha[0]), float(alpha[1]), int(bool(rest)), gp, gld,
                ws.buf.data_ptr(), ws.nbytes)
        self.workspace = ws
        self._set("dspark_distill_grad", args, stream, out, (logits, teacher_ids, teacher_logp, norm, grad_loss, ws),
                  dev)


def distill_grad(logits, teacher_ids, teacher_logp, norm, grad_loss, *, T=1.0, alpha=(1.0, 0.0), rest=True,
                 workspace=None, stream=None, out=None):
    """Gradient of ``distill_loss``'s loss (of weight 1) with respect to the logits, in their dtype, times
    ``grad_loss`` [...] fp32, from the forward call's ``norm``.  ``out`` may be the logits themselves.  See
    ``dspark_distill_grad``."""
    return DistillGradPlan(logits, teacher_ids, teacher_logp, norm, grad_loss, T=T, alpha=alpha, rest=rest,
                           workspace=workspace, stream=stream, out=out).run()


class CapacityRing:
    """The steps/s table the prefix scheduler reads, delayed by ``delay`` steps.

    "DSpark：既要猜得连贯…" ("设计") notes that the production scheduler uses a capacity
    estimate delayed by two steps, to fit asynchronous scheduling and CUDA Graphs.  ``table`` is
    one fixed device buffer that ``prefix_schedule`` can read (also from a captured graph);
    ``advance(sps)`` records this step's measured table and copies the one recorded ``delay``
    steps earlier into ``table``, stream-ordered (until ``delay`` steps have been recorded,
    ``table`` keeps the initial table).  Only tensor copies: no arithmetic of the method here.
    """

    def __init__(self, initial, delay: int = 2):
        if delay < 0:
            raise ValueError("delay must be >= 0")
        self.delay = delay
        self.table = initial.clone()
        self._ring = [torch.empty_like(initial) for _ in range(delay + 1)]
        self._step = 0

    def advance(self, sps) -> "torch.Tensor":
        slot = self._step % (self.delay + 1)
        self._ring[slot].copy_(sps, non_blocking=True)
        if self._step >= self.delay:
            self.table.copy_(self._ring[(self._step - self.delay) % (self.delay + 1)], non_blocking=True)
        self._step += 1
        return self.table


def draft_path(head: int, B: int, V: int, r: int, bf16: bool = True) -> int:
    return _lib.load().dspark_draft_path(head, B, V, r, _BF16 if bf16 else _F32)


def draft_launches(head: int, B: int, V: int, r: int, bf16: bool = True) -> int:
    return _lib.load().dspark_draft_launches(head, B, V, r, _BF16 if bf16 else _F32)


def draft_cluster(head: int, B: int, V: int, r: int, bf16: bool = True) -> int:
    """Blocks per thread-block cluster of the draft kernel these arguments select (1: none)."""
    return _lib.load().dspark_draft_cluster(head, B, V, r, _BF16 if bf16 else _F32)


def draft_loss_launches(B: int, gamma: int, V: int, with_grad: bool = True) -> int:
    """Kernel launches of one draft_loss call (the sub-batch pipeline and the totals)."""
    return _lib.load().dspark_draft_loss_launches(B, gamma, V, int(with_grad))
