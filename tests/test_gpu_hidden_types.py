"""Autograd of the norm for every mix of types, against float64 gradients of the inputs as they are.

Tolerances, u = 2^-24: as in test_gpu_hidden.py; a gradient is computed from h as it is kept (fp32 where x or the
residual is: one rounding, u of h, else bf16: 2^-9 of its power of two, at most 2^-8 of h) and rounded once to the
input's type.  With e that rounding's bound and rstd within 52 u: xh = h rstd moves by (e + 52 u), so
  dx:  rstd |g w| 60 u + rstd |xh| mean|g w xh| (102 u + 2 (e + 52 u) + 52 u), and half a step of its type;
  dweight: (R + 3) u + e + 52 u of the sum of |g xh|, and half a step."""
import pytest
import torch

from test_gpu_hidden import B, device_status_stays_clear  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
F, H = torch.float32, torch.bfloat16


@pytest.mark.parametrize("R,d", [(1, 8), (90, 264), (300, 1001)])
@pytest.mark.parametrize("x,res,out", [(F, H, F), (F, H, H), (F, F, F), (H, F, H), (H, F, F), (H, H, H), (F, None, H)])
def test_gradients_of_every_mix(B, R, d, x, res, out):
    from denoising_sampler_step_gb300 import training as T
    g = torch.Generator(device="cuda").manual_seed(R)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    xt = rnd(R, d).to(x).requires_grad_(True)
    rt = rnd(R, d).to(res).requires_grad_(True) if res else None
    w = rnd(d).requires_grad_(True)
    y, h = T.rms_norm(xt, w, residual=rt, eps=1e-3, weight_offset=1.0, dtype=out)
    assert y.dtype == out and (h is None if res is None else h.dtype == res)
    up, uh = rnd(R, d).to(out), rnd(R, d).to(res) if res else None
    leaves = [xt, w] + ([rt] if res else [])
    got = torch.autograd.grad([y] + ([h] if res else []), leaves, [up] + ([uh] if res else []))
    assert [t.dtype for t in got] == [t.dtype for t in leaves]

    wide = [t.detach().double().requires_grad_(True) for t in leaves]
    hd = wide[0] if res is None else wide[0] + wide[2]
    rstd = (hd.square().mean(1, keepdim=True) + 1e-3) ** -0.5
    yd = hd * rstd * (1 + wide[1])
    ref = torch.autograd.grad([yd] + ([hd] if res else []), wide, [up.double()] + ([uh.double()] if res else []))
    e = 0.0 if res is None else U if F in (x, res) else 2.0 ** -8
    with torch.no_grad():
        gw, xh = (up.double() * (1 + wide[1])).abs(), (hd * rstd).abs()
        tol = rstd * (60 * U * gw + (258 * U + 2 * e) * xh * (gw * xh).mean(1, keepdim=True))
        if res:
            tol = tol + 2 * U * uh.double().abs()
        terms = (up.double().abs() * xh).sum(0)
    for a, b in [(got[0], ref[0])] + ([(got[2], ref[2])] if res else []):
        assert ((a - b).abs() <= tol + (HALF[a.dtype] + 2 * U) * b.abs()).all()
    assert ((got[1] - ref[1]).abs() <= ((R + 55) * U + e) * terms + U * ref[1].abs()).all()
    # h itself: one rounding
    if res:
        assert ((h - hd).abs() <= (HALF[res] + U) * hd.abs()).all()


def test_nothing_else_changes_with_the_mix(B):
    """The outputs are those of the call itself, whichever matrix is in fp32."""
    from denoising_sampler_step_gb300 import training as T
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r = torch.randn(50, 264, generator=g, device="cuda"), torch.randn(50, 264, generator=g, device="cuda").bfloat16()
    o = B.dg_rms_norm(x, residual=r)
    y, h = T.rms_norm(x, residual=r)
    assert torch.equal(y, o["out"]) and torch.equal(h, o["hidden"]) and h.dtype == H
