"""Host-side refusals of the calls that process logits and distil from top log probabilities: every bad
argument is found before anything is enqueued, so these run without a GPU."""
import ctypes

import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

P = ctypes.c_void_p(1 << 20)
Q = ctypes.c_void_p(1 << 30)
G = ctypes.c_void_p(1 << 32)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from semi_autoregressive_drafting_gb300 import _build, _lib
    _build.build()
    return _lib.load()


def at(n):
    return ctypes.c_void_p(n)


BAD = [dict(B=-1), dict(R=0), dict(R=33), dict(V=1), dict(V=(1 << 24) + 1), dict(B=1 << 22, R=8), dict(idt=2),
       dict(odt=5), dict(ld=99), dict(old=99), dict(H=-1), dict(H=(1 << 24) + 1), dict(h=None), dict(hld=7),
       dict(mld=3), dict(M=0), dict(mask=None), dict(rows=None, M=7), dict(z=None), dict(out=None),
       dict(z=at((1 << 20) + 2)), dict(out=at((1 << 30) + 1)), dict(mask=at(6)), dict(h=at(2)),
       # overlapping without being the same rows of the same type
       dict(out=at((1 << 20) + 4)), dict(out=P, old=104), dict(out=P, odt=1), dict(out=at((1 << 20) - 400))]


def process(lib, B=4, R=2, V=100, idt=0, z=P, ld=100, h=P, hld=8, H=8, nb=0, bt=None, b=None, mask=P, mld=4, M=8, rows=P,
            odt=0, out=Q, old=100):
    return lib.dspark_process_logits(B, R, V, idt, z, ld, h, hld, H, None, None, None, P, None, None, nb, bt, b, mask,
                                     mld, M, rows, odt, out, old, None)


def test_process_refusals(lib):
    assert process(lib, B=0) == 0
    for kw in BAD + [dict(nb=-1), dict(nb=1025), dict(nb=3), dict(nb=3, bt=P)]:
        assert process(lib, **kw) == 1, kw
        assert lib.dspark_last_error()


def test_process_grad_refusals(lib):
    def call(B=4, R=2, V=100, idt=0, z=G, ld=100, h=P, hld=8, H=8, mask=P, mld=4, M=8, rows=P, odt=0, out=Q, old=100,
             rep=P, raw=P, rld=100):
        return lib.dspark_process_logits_grad(B, R, V, idt, z, ld, odt, raw, rld, h, hld, H, None, None, None, rep,
                                              mask, mld, M, rows, out, old, None)
    assert call(B=0) == 0
    for kw in BAD:
        kw = {**kw}
        if "out" in kw and kw["out"] is not None and kw["out"].value < 1 << 30:
            kw["z"] = P
        assert call(**kw) == 1, kw
    for kw in [dict(raw=None), dict(rld=99), dict(raw=at(2)), dict(out=P), dict(out=at((1 << 20) + 200))]:
        assert call(**kw) == 1, kw


def test_distill_refusals(lib):
    def loss(N=4, V=100, T=1.0, dt=0, z=P, ld=100, K=5, ids=P, lq=P, w=P, a=1.0, b=0.0, out=P, parts=P, norm=P, g=Q,
             gld=100, ws=P, nb=BIG):
        return lib.dspark_distill_loss(N, V, T, dt, z, ld, K, ids, lq, w, a, b, 1, out, parts, norm, g, gld, ws, nb,
                                       None)

    def grad(N=4, V=100, T=1.0, dt=0, z=P, ld=100, K=5, ids=P, lq=P, w=P, a=1.0, b=0.0, norm=P, g=Q, gld=100, ws=P,
             nb=BIG):
        return lib.dspark_distill_grad(N, V, T, dt, z, ld, K, ids, lq, norm, w, a, b, 1, g, gld, ws, nb, None)
    bad = [dict(N=-1), dict(N=(1 << 24) + 1), dict(V=1), dict(T=0.0), dict(T=float("nan")), dict(T=1e-45), dict(dt=2),
           dict(ld=99), dict(gld=99), dict(K=0), dict(K=129), dict(V=4, ld=100, K=5), dict(z=None), dict(ids=None),
           dict(lq=None), dict(a=float("inf")), dict(b=float("nan")), dict(z=at((1 << 20) + 2)), dict(g=at(6)),
           dict(norm=at(8)), dict(g=at((1 << 20) + 40)), dict(g=P, gld=101)]
    for call in (loss, grad):
        assert call(N=0) == 0
        for kw in bad:
            assert call(**kw) == 1, kw
            assert lib.dspark_last_error()
        for kw in [dict(ws=None), dict(ws=at(264)), dict(nb=100)]:
            assert call(**kw) == 2, kw
    assert loss(out=None, parts=None, norm=None, g=None) == 1
    assert loss(parts=at(4)) == 1
    for kw in [dict(norm=None), dict(w=None), dict(g=None)]:
        assert grad(**kw) == 1, kw
    for args in [(-1, 100, 5), (4, 1, 1), (4, 100, 0), (4, 100, 129), (4, 3, 4), (1 << 24, 1 << 24, 5)]:
        assert lib.dspark_distill_workspace_bytes(*args) == 0
    assert lib.dspark_distill_workspace_bytes(0, 100, 5) > 0


def test_plans_refuse_host_tensors():
    z, i, q = torch.zeros(2, 10), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    for call in (lambda: ds.process_logits(z), lambda: ds.process_logits_grad(z, z), lambda: ds.distill_loss(z, i, q),
                 lambda: ds.distill_grad(z, i, q, torch.zeros(2, 4), torch.zeros(2))):
        with pytest.raises(ValueError):
            call()


class _Cuda(torch.Tensor):
    """A host tensor that says it is on the GPU: the checks of shapes, types and strides alone."""
    is_cuda = True

    @property
    def device(self):
        return torch.device("cuda", 0)


def cu(t):
    return t.as_subclass(_Cuda)


@pytest.fixture
def on_gpu(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    from contextlib import nullcontext
    monkeypatch.setattr(torch.cuda, "stream", lambda s: nullcontext())


def test_process_plan_refuses_shapes_types_and_strides(on_gpu):
    z = cu(torch.zeros(3, 2, 40))
    out = cu(torch.zeros(3, 2, 40))
    h = cu(torch.zeros(3, 8, dtype=torch.int32))
    i3, f3 = cu(torch.zeros(3, dtype=torch.int32)), cu(torch.zeros(3))
    m = cu(torch.zeros(6, 2, dtype=torch.int32))
    value = [dict(history=cu(torch.zeros(2, 8, dtype=torch.int32))), dict(history=cu(torch.zeros(8, 3, dtype=torch.int32).t())),
             dict(lengths=i3), dict(history=h, lengths=cu(torch.zeros(2, dtype=torch.int32))),
             dict(drafted=cu(torch.zeros(3, 2, dtype=torch.int32))), dict(repetition=cu(torch.zeros(4))),
             dict(bias=cu(torch.zeros(3, 2))), dict(bias=cu(torch.zeros(3, 2)), bias_tokens=cu(torch.zeros(3, 1, dtype=torch.int32))),
             dict(mask=cu(torch.zeros(6, 1, dtype=torch.int32))), dict(mask=cu(torch.zeros(5, 2, dtype=torch.int32))),
             dict(mask_rows=cu(torch.zeros(3, 2, dtype=torch.int32))),
             dict(mask=m, mask_rows=cu(torch.zeros(3, dtype=torch.int32))),
             dict(mask=cu(torch.zeros(2, 6, dtype=torch.int32).t())), dict(out=cu(torch.zeros(3, 40)))]
    types = [dict(history=cu(torch.zeros(3, 8))), dict(history=h, lengths=cu(torch.zeros(3))), dict(presence=i3),
             dict(mask=cu(torch.zeros(6, 2))), dict(bias=cu(torch.zeros(3, 2)), bias_tokens=cu(torch.zeros(3, 2)))]
    for kw in value:
        with pytest.raises(ValueError):
            ds.ProcessPlan(z, **{"out": out, **kw})
    for kw in types:
        with pytest.raises(TypeError):
            ds.ProcessPlan(z, **{"out": out, **kw})
    with pytest.raises(ValueError):
        ds.ProcessPlan(cu(torch.zeros(40)), out=cu(torch.zeros(40)))
    with pytest.raises(ValueError):
        ds.ProcessGradPlan(cu(torch.zeros(3, 2, 41)), z, out=out)
    with pytest.raises(ValueError):
        ds.ProcessGradPlan(z, z, out=cu(torch.zeros(3, 2, 40, dtype=torch.bfloat16)))


def test_distill_plan_refuses_shapes_and_types(lib, on_gpu):
    z, i, q = cu(torch.zeros(4, 40)), cu(torch.zeros(4, 3, dtype=torch.int32)), cu(torch.zeros(4, 3))
    f = lambda *s: cu(torch.zeros(*s))
    ws = ds.DistillWorkspace.__new__(ds.DistillWorkspace)
    ws.buf, ws.nbytes = f(8), 1 << 30
    out = ds.DistillOutput(f(4), f(4, 2), f(4, 4), f(4, 40))
    kw = dict(workspace=ws, out=out)
    for a in [(z, cu(torch.zeros(3, 3, dtype=torch.int32)), q), (z, i, f(4, 2)), (z[:, :1], i, q)]:
        with pytest.raises(ValueError):
            ds.DistillPlan(*a, **kw)
    with pytest.raises(TypeError):
        ds.DistillPlan(z, q, q, **kw)
    with pytest.raises(ValueError):
        ds.DistillPlan(z, i, q, **{**kw, "weight": f(5)})
    with pytest.raises(ValueError):
        ds.DistillPlan(z, i, q, **{**kw, "out": ds.DistillOutput(f(4), f(4, 2), f(4, 4), None)})
    with pytest.raises(ValueError):
        ds.DistillPlan(z, i, q, **{**kw, "out": ds.DistillOutput(f(4), f(4, 2), f(4, 2), f(4, 40))})
    for n, g in [(f(4, 2), f(4)), (f(4, 4), f(3)), (None, f(4)), (f(4, 4), None)]:
        with pytest.raises(ValueError):
            ds.DistillGradPlan(z, i, q, n, g, workspace=ws, out=f(4, 40))


def test_no_request_needs_no_arrays(lib):
    """Empty arrays have no address; a call without requests does nothing."""
    assert process(lib, B=0, z=None, out=None, h=None, hld=0, nb=3, mask=None, rows=None) == 0
    assert process(lib, B=0, M=0, rows=None) == 0
    assert process(lib, B=0, R=33) == 1
