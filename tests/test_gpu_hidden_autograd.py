"""The denoising run's gradients against float64's, and the transforms that the autograd functions do not have."""
import pytest
import torch

from denoising_sampler_step_gb300 import inputs
from test_gpu_hidden import B, device_status_stays_clear  # noqa: F401

pytestmark = pytest.mark.gpu


def test_the_denoising_runs_gradients(B):
    """Table (as embedding and as head) and norm weight.  Tolerance: a logit's fp32 sum of d = 256 terms is off by at most
    256 2^-24 of their magnitudes, sum |y| |W| of some 16 (y of order 1, W of 1 / 16): 2.5e-4, and a probability by twice
    that; what multiplies it is exact to 1e-5.  So 1e-3 of the gradient's magnitudes, taken as its largest entry per row and
    what rounding leaves of the rest."""
    from denoising_sampler_step_gb300 import finetune
    wl = inputs.WORKLOADS["tiny"]
    V, d, R = wl.V, wl.d, 4 * wl.R
    g = torch.Generator(device="cuda").manual_seed(1)
    table = (torch.randn(V, d, generator=g, device="cuda") / d ** 0.5).requires_grad_(True)
    weight = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).requires_grad_(True)
    clean = torch.randint(V - 1, (R,), generator=g, device="cuda").int()
    signal = 0.1 * torch.randn(R, d, generator=g, device="cuda")
    noised = torch.where(torch.rand(R, generator=g, device="cuda") < 0.3, V - 1, clean).int()   # V - 1 occurs as an input alone
    noised[-wl.R // 4:] = -1
    assert (noised == V - 1).any() and not (clean == V - 1).any()
    loss = finetune.denoising_loss(table, weight, noised, clean, signal, wl.gamma)
    got = torch.autograd.grad(loss, (table, weight))

    W, w = (t.detach().double().requires_grad_(True) for t in (table, weight))
    on = noised >= 0
    x = torch.where(on[:, None], wl.gamma * W[noised.clamp(min=0).long()], 0.0) + signal.double()
    y = x * (x.square().mean(1, keepdim=True) + 1e-6) ** -0.5 * w
    logp = torch.log_softmax(y @ W.T, 1).gather(1, clean.long()[:, None])[:, 0]
    ref = -logp[on].sum() / on.sum()
    assert abs(float(loss) - float(ref)) <= 1e-3
    want = torch.autograd.grad(ref, (W, w))
    for a, b in zip(got, want):
        b2, a2 = (t.view(-1, d) for t in (b, a.double()))
        assert ((a2 - b2).abs() <= 1e-3 * b2.abs().amax(1, keepdim=True) + 1e-6 * b2.abs().max()).all()
    # the mask token's row, and the weight, have gradients of their own and of the right sign and size
    for a, b in ((got[0][V - 1], want[0][V - 1]), (got[1], want[1])):
        assert b.abs().max() > 0
        assert torch.nn.functional.cosine_similarity(a.double(), b, dim=0) > 0.9999
        assert float(a.double().norm() / b.norm()) == pytest.approx(1.0, abs=1e-3)


def test_transforms_are_refused(B):
    from denoising_sampler_step_gb300 import training as T
    x, w = torch.randn(4, 16, device="cuda"), torch.randn(16, device="cuda")
    tok = torch.arange(4, dtype=torch.int32, device="cuda")
    for f in (lambda t: T.rms_norm(t, w)[0], lambda t: T.token_embed(t, tok, 2.0)):
        with pytest.raises((RuntimeError, NotImplementedError)):
            torch.func.jvp(f, (x,), (x,))
        with pytest.raises((RuntimeError, NotImplementedError)):
            torch.autograd.forward_ad.unpack_dual(dual(f, x))
        with pytest.raises((RuntimeError, NotImplementedError)):
            torch.func.vmap(f)(x.expand(3, 4, 16))
        with pytest.raises((RuntimeError, NotImplementedError)):
            torch.func.grad(lambda t: f(t).sum())(x)


def dual(f, x):
    with torch.autograd.forward_ad.dual_level():
        return f(torch.autograd.forward_ad.make_dual(x, torch.ones_like(x)))
