"""Host-side refusals of the token, table and bias-gradient calls: every bad argument is found before
anything is enqueued, so these run without a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from semi_autoregressive_drafting_gb300 import _build, _lib
    _build.build()
    return _lib.load()


P = ctypes.c_void_p(256)
BIG = 1 << 40


def test_token_logprobs_refusals(lib):
    def call(N=4, V=100, T=1.0, dt=0, z=P, ld=100, tok=P, top=2, logp=P, norm=P, ids=P, ws=P, nb=BIG):
        return lib.dspark_token_logprobs(N, V, T, dt, z, ld, tok, top, logp, norm, P, P, ids, P, ws, nb, None)
    assert call(N=0) == 0
    for kw in [dict(N=-1), dict(V=1), dict(V=(1 << 24) + 1), dict(T=0.0), dict(T=float("nan")),
               dict(T=float("inf")), dict(T=1e-45), dict(dt=2), dict(ld=99), dict(z=None), dict(tok=None),
               dict(top=-1), dict(top=33), dict(V=8, ld=8, top=9), dict(ids=None),
               dict(z=ctypes.c_void_p(258)), dict(norm=ctypes.c_void_p(260))]:
        assert call(**kw) == 1, kw
        assert lib.dspark_last_error()
    for kw in [dict(ws=None), dict(ws=ctypes.c_void_p(264)), dict(nb=0)]:
        assert call(**kw) == 2, kw
    for args in [(-1, 100, 0), (1, 1, 0), (1, 100, 33), (1, 8, 9)]:
        assert lib.dspark_token_logprobs_workspace_bytes(*args) == 0
    assert lib.dspark_token_logprobs_workspace_bytes(0, 100, 0) > 0


def test_token_logprobs_grad_refusals(lib):
    def call(N=4, V=100, T=1.0, dt=0, z=P, ld=100, tok=P, norm=P, ent=P, gl=P, gh=P, out=P, gld=100):
        return lib.dspark_token_logprobs_grad(N, V, T, dt, z, ld, tok, norm, ent, gl, gh, out, gld, None)
    assert call(N=0) == 0
    for kw in [dict(N=-1), dict(V=1), dict(T=-1.0), dict(dt=7), dict(ld=1), dict(gld=99), dict(z=None),
               dict(norm=None), dict(out=None), dict(gl=None, gh=None), dict(tok=None), dict(ent=None),
               dict(out=ctypes.c_void_p(257))]:
        assert call(**kw) == 1, kw


def test_embedding_refusals(lib):
    def call(N=4, V=10, D=8, scale=1.0, wdt=0, W=P, tok=P, odt=0, out=P):
        return lib.dspark_embedding(N, V, D, scale, wdt, W, tok, odt, out, None)
    assert call(N=0) == 0
    for kw in [dict(N=-1), dict(V=0), dict(D=0), dict(scale=float("inf")), dict(wdt=3), dict(odt=-1),
               dict(W=None), dict(tok=None), dict(out=None), dict(W=ctypes.c_void_p(258))]:
        assert call(**kw) == 1, kw

    def grad(N=4, V=10, D=8, scale=1.0, gdt=0, g=P, tok=P, odt=0, out=P, acc=0, ws=P, nb=BIG):
        return lib.dspark_embedding_grad(N, V, D, scale, gdt, g, tok, odt, out, acc, ws, nb, None)
    for kw in [dict(N=-1), dict(N=(1 << 24) + 1), dict(V=0), dict(D=0), dict(scale=float("nan")), dict(gdt=2),
               dict(odt=2), dict(g=None), dict(tok=None), dict(out=None), dict(out=ctypes.c_void_p(257))]:
        assert grad(**kw) == 1, kw
    for kw in [dict(ws=None), dict(ws=ctypes.c_void_p(16)), dict(nb=8)]:
        assert grad(**kw) == 2, kw
    assert lib.dspark_embedding_grad_workspace_bytes(-1, 10, 8) == 0
    assert lib.dspark_embedding_grad_workspace_bytes(0, 10, 8) > 0


def test_bias_grad_refusals(lib):
    def call(N=4, V=100, r=16, gdt=0, G=P, wdt=1, a=P, W2=P, lay=0, ga=P, gw=P):
        return lib.dspark_bias_grad(N, V, r, gdt, G, wdt, a, W2, lay, ga, gw, 0, P, BIG, None)
    for kw in [dict(N=-1), dict(V=1), dict(r=12), dict(r=0), dict(r=520), dict(gdt=2), dict(wdt=2), dict(lay=2),
               dict(G=None), dict(a=None), dict(W2=None), dict(ga=None, gw=None),
               dict(G=ctypes.c_void_p(260)), dict(gw=ctypes.c_void_p(264))]:
        assert call(**kw) == 1, kw
    assert lib.dspark_bias_grad_workspace_bytes(4, 100, 12, 1) == 0
