"""What the hidden stream's calls refuse, on the host (no GPU): nothing is launched for these."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
A, Bq, C, D, E, F = (P(i << 44) for i in range(1, 7))    # addresses far apart, never read
WS = 1 << 40
INV, UNS = 1, 2


@pytest.fixture(scope="module")
def L():
    from denoising_sampler_step_gb300 import build
    build.build()
    from denoising_sampler_step_gb300 import binding
    return binding.lib


def off(p, n):
    return P(p.value + n)


def embed(L, table=A, dtype=1, scale=None, V=100, s=0, e=100, rows=100, ldw=16, d=16, token=Bq, R=4, out=C, odt=1,
          ldo=16):
    return L.dg_token_embed(table, dtype, scale, V, s, e, rows, ldw, d, token, R, 1.0, out, odt, ldo, None)


def test_token_embed(L):
    for kw in (dict(R=-1), dict(d=0), dict(V=0), dict(s=-1), dict(s=60, e=40), dict(e=101), dict(rows=99), dict(ldw=15),
               dict(ldo=15), dict(token=None), dict(table=None), dict(out=None), dict(dtype=3), dict(dtype=-1),
               dict(odt=2), dict(dtype=2), dict(scale=D), dict(out=off(A, 32)), dict(out=off(Bq, 8))):
        assert embed(L, **kw) == INV, kw
    for kw in (dict(V=2 ** 31, rows=2 ** 31), dict(R=2 ** 28 + 1), dict(d=2 ** 30, ldw=2 ** 30, ldo=2 ** 30),
               dict(table=off(A, 1)), dict(out=off(C, 1)), dict(odt=0, out=off(C, 2)), dict(token=off(Bq, 2)),
               dict(dtype=2, scale=off(D, 1)), dict(ldo=1 << 60)):
        assert embed(L, **kw) == UNS, kw
    assert b"out" in L.dg_last_error()
    assert embed(L, R=0, token=None, out=None, table=None) == 0


def backward(L, grad=A, dtype=1, R=4, d=16, ldg=16, token=Bq, V=100, s=0, e=100, table=C, tdt=0, rows=100, ldt=16,
             acc=0, ws=D, n=WS):
    return L.dg_token_embed_backward(grad, dtype, R, d, ldg, token, V, s, e, 1.0, table, tdt, rows, ldt, acc, ws, n, None)


def test_token_embed_backward(L):
    need = L.dg_token_embed_backward_workspace_size(4, 100, 16)
    assert need > 0
    for kw in (dict(R=-1), dict(d=0), dict(s=5, e=4), dict(rows=99), dict(ldg=15), dict(ldt=15), dict(dtype=2),
               dict(tdt=2), dict(token=None), dict(grad=None), dict(table=None), dict(ws=None), dict(n=need - 1),
               dict(table=off(A, 64)), dict(table=Bq), dict(ws=C), dict(ws=A), dict(ws=Bq)):
        assert backward(L, **kw) == INV, kw
    for kw in (dict(ws=off(D, 8)), dict(token=off(Bq, 1)), dict(grad=off(A, 1)), dict(table=off(C, 2)), dict(V=2 ** 31, e=2 ** 31, rows=2 ** 31)):
        assert backward(L, **kw) == UNS, kw
    # nothing to do
    assert backward(L, R=0, acc=1, token=None, grad=None, ws=None, n=0) == 0
    assert backward(L, s=7, e=7, table=None) == 0
    for bad in ((0, 100, 16), (-1, 100, 16), (4, -1, 16), (4, 100, 0), (2 ** 28 + 1, 100, 16), (4, 2 ** 31, 16)):
        assert L.dg_token_embed_backward_workspace_size(*bad) == 0, bad


def norm(L, x=A, dtype=1, R=4, d=16, ldx=16, res=None, rdt=1, ldr=16, w=None, wdt=0, offset=0.0, eps=1e-6, hid=None,
         hdt=1, ldh=16, out=C, odt=1, ldo=16, scale=None, rstd=D):
    return L.dg_rms_norm(x, dtype, R, d, ldx, res, rdt, ldr, w, wdt, offset, eps, hid, hdt, ldh, out, odt, ldo, scale,
                         rstd, None)


def test_rms_norm(L):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(R=-1), dict(d=0), dict(ldx=15), dict(res=Bq, ldr=15), dict(hid=Bq, ldh=15), dict(ldo=15), dict(x=None),
               dict(out=None), dict(dtype=2), dict(res=Bq, rdt=2), dict(hid=Bq, hdt=2), dict(odt=3), dict(w=E, wdt=2),
               dict(w=E, wdt=-1), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(offset=nan), dict(offset=inf),
               dict(odt=2), dict(scale=E), dict(out=off(A, 2)), dict(out=A, odt=0), dict(out=A, ldo=24),
               dict(hid=C), dict(hid=off(A, 2)), dict(res=Bq, hid=off(Bq, 2)), dict(res=Bq, out=off(Bq, 4)),
               dict(w=C, wdt=1), dict(rstd=A), dict(rstd=C), dict(odt=2, scale=D), dict(rstd=off(D, 4), odt=2, scale=D)):
        assert norm(L, **kw) == INV, kw
    for kw in (dict(R=2 ** 28 + 1), dict(d=32769, ldx=32769, ldo=32769), dict(x=off(A, 1)), dict(out=off(C, 1)),
               dict(w=off(E, 2)), dict(res=off(Bq, 2), rdt=0), dict(rstd=off(D, 2)), dict(odt=2, scale=off(E, 1))):
        assert norm(L, **kw) == UNS, kw
    assert norm(L, R=0, x=None, out=None, rstd=None) == 0


def norm_back(L, grad=A, dtype=1, R=4, d=16, ldg=16, hid=Bq, hdt=1, ldh=16, rstd=D, w=None, wdt=0, offset=0.0, up=None,
              udt=1, ldu=16, gx=C, ldx=16, gw=None, ws=F, n=WS):
    return L.dg_rms_norm_backward(grad, dtype, R, d, ldg, hid, hdt, ldh, rstd, w, wdt, offset, up, udt, ldu, gx, ldx,
                                  gw, ws, n, None)


def test_rms_norm_backward(L):
    W, G = P(1 << 55), P(1 << 54)
    for kw in (dict(R=-1), dict(d=0), dict(ldg=15), dict(ldh=15), dict(up=E, ldu=15), dict(ldx=15), dict(grad=None),
               dict(hid=None), dict(gx=None), dict(rstd=None), dict(dtype=2), dict(hdt=2), dict(up=E, udt=2),
               dict(w=W, wdt=2), dict(gw=G), dict(gx=off(A, 2)), dict(gx=A, dtype=0), dict(gx=Bq, ldx=24),
               dict(up=E, gx=off(E, 2)), dict(gx=D), dict(w=W, gw=W), dict(w=W, gw=A), dict(w=C), dict(w=W, gw=D)):
        assert norm_back(L, **kw) == INV, kw
    for kw in (dict(d=32769, ldg=32769, ldh=32769, ldx=32769), dict(grad=off(A, 1)), dict(w=W, gw=off(G, 2)),
               dict(w=off(W, 1), wdt=1), dict(rstd=off(D, 3))):
        assert norm_back(L, **kw) == UNS, kw
    assert norm_back(L, R=0, grad=None, hid=None, rstd=None, gx=None) == 0
    assert L.dg_rms_norm_backward_workspace_size(4, 32769) == 0 == L.dg_rms_norm_backward_workspace_size(0, 16)


def head(L, X=A, ldx=16, xs=Bq, R=4, d=16, Q=C, s=D, V=100, ldq=16, out=E, dtype=0, ldl=100):
    return L.dg_head_e4m3(X, ldx, xs, R, d, Q, s, V, ldq, out, dtype, ldl, None)


def test_head(L):
    for kw in (dict(R=-1), dict(d=0), dict(V=0), dict(ldx=15), dict(ldq=15), dict(ldl=99), dict(X=None), dict(Q=None),
               dict(out=None), dict(xs=None), dict(s=None), dict(dtype=2), dict(out=A), dict(out=off(Bq, -16)),
               dict(out=off(C, 16)), dict(out=D)):
        assert head(L, **kw) == INV, kw
    for kw in (dict(R=2 ** 28 + 1), dict(V=2 ** 31, ldl=2 ** 31), dict(d=2 ** 24, ldx=2 ** 24, ldq=2 ** 24), dict(ldx=24),
               dict(ldq=40), dict(X=off(A, 8)), dict(Q=off(C, 8)), dict(out=off(E, 8)), dict(xs=off(Bq, 2)), dict(s=off(D, 1)), dict(V=99, ldl=99),
               dict(dtype=1, ldl=100)):
        assert head(L, **kw) == UNS, kw
    assert b"multiple of 8 elements" in L.dg_last_error()
    assert head(L, R=0, X=None, xs=None, out=None, Q=None) == 0


def test_the_binding_wants_the_gpu():
    from denoising_sampler_step_gb300 import binding as B, training
    x, tok = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    codes = torch.zeros(2, 8, dtype=torch.uint8)
    for call in (lambda: B.dg_token_embed(x, tok), lambda: B.dg_token_embed_backward(x, tok, 4),
                 lambda: B.dg_rms_norm(x), lambda: B.dg_rms_norm_backward(x, x, x[:, 0]),
                 lambda: B.dg_head_e4m3(codes, x[:, 0], codes, x[:, 0])):
        with pytest.raises(ValueError, match="must be on the GPU"):
            call()
    with pytest.raises(TypeError, match="8-bit"):
        training.rms_norm(x, dtype=torch.uint8)
