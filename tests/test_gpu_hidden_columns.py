"""Matrices that are different columns of one buffer: they share its rows but no entry, and each call gives what it
gives on matrices apart.  Tolerances, u = 2^-24: two results of the same formula are each within those of
test_gpu_hidden.py, 56 u and a step of the type of the largest entry for the norm, twice 102 u for its gradient, whose
weight's is (R + 3) u of the terms' magnitudes, twice."""
import pytest
import torch

from test_gpu_hidden import B, device_status_stays_clear  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def columns(kind, R, d, n, g=None, gap=0):
    """n matrices [R, d] beside one another, `gap` columns between them."""
    buf = torch.full((R, n * (d + gap)), 7.0, device="cuda", dtype=kind)
    views = [buf[:, i * (d + gap):i * (d + gap) + d] for i in range(n)]
    if g is not None:
        for v in views:
            v.copy_(torch.randn(R, d, generator=g, device="cuda"))
    return views


@pytest.mark.parametrize("R,d,gap", [(1, 5, 0), (2, 8, 0), (40, 264, 0), (40, 264, 8), (700, 33, 0), (33, 999, 3), (5003, 264, 0)])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_norm_and_its_gradient(B, R, d, gap, kind):
    g = torch.Generator(device="cuda").manual_seed(R)
    x, r, y, h, dx = columns(kind, R, d, 5, g, gap)
    w = torch.randn(d, generator=g, device="cuda")
    apart = [t.contiguous() for t in (x, r)]
    want = B.dg_rms_norm(apart[0], w, residual=apart[1])
    o = B.dg_rms_norm(x, w, residual=r, out={"out": y, "hidden": h})
    step = torch.finfo(kind).eps
    for a, b in ((y, want["out"]), (h, want["hidden"])):
        assert (a.double() - b.double()).abs().max() <= (step + 112 * U) * b.double().abs().max()
    n = B.dg_rms_norm_backward(y, h, o["rstd"], w, grad_hidden=r, out={"grad": dx})
    m = B.dg_rms_norm_backward(y.contiguous(), h.contiguous(), o["rstd"], w, grad_hidden=r.contiguous())
    xh = h.double() * o["rstd"].double()[:, None]
    gw = (y.double() * w.double()).abs()
    size = (o["rstd"].double()[:, None] * (gw + xh.abs() * (gw * xh.abs()).mean(1, keepdim=True)) + r.double().abs()).max()
    assert (n["grad"].double() - m["grad"].double()).abs().max() <= (step + 204 * U) * size
    terms = (y.double() * xh).abs().sum(0)
    assert ((n["grad_weight"] - m["grad_weight"]).abs() <= 2 * (R + 3) * U * terms).all()
    assert torch.equal(x, apart[0]) and torch.equal(r, apart[1])


@pytest.mark.parametrize("d", [8, 33, 264])
def test_lookup_and_its_gradient(B, d):
    g = torch.Generator(device="cuda").manual_seed(d)
    W, out, grad = columns(torch.float32, 500, d, 3, g)
    tok = torch.randint(500, (500,), generator=g, device="cuda").int()
    B.dg_token_embed(W, tok, 2.0, out=out)
    assert torch.equal(out, 2.0 * W[tok.long()])
    before = W.contiguous()
    B.dg_token_embed_backward(out, tok, 500, 1.0, out=grad)
    want = torch.zeros(500, d, dtype=torch.float64, device="cuda").index_add_(0, tok, out.double())
    size = torch.zeros(500, d, dtype=torch.float64, device="cuda").index_add_(0, tok, out.double().abs())
    assert ((grad - want).abs() <= 503 * U * size).all()
    assert torch.equal(W, before)


def test_columns_that_do_overlap_are_refused(B):
    buf = torch.zeros(20, 64, device="cuda")
    for a, b in ((0, 1), (0, 31), (31, 0), (16, 32)):
        with pytest.raises(B.DgError, match="overlaps"):
            B.dg_rms_norm(buf[:, a:a + 32], out={"out": buf[:, b:b + 32]})
    # one that reaches into the next row of the other
    flat = torch.zeros(20 * 64 + 64, device="cuda")
    x, y = flat[:20 * 64].view(20, 64)[:, :32], flat[40:40 + 20 * 64].view(20, 64)[:, :32]
    with pytest.raises(B.DgError, match="overlaps"):
        B.dg_rms_norm(x, out={"out": y})
    with pytest.raises(B.DgError, match="overlaps"):
        B.dg_rms_norm(y, out={"out": x})
