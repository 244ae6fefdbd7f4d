"""The differentiable losses inside autograd expressions, and the small training run."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    from denoising_sampler_step_gb300 import build
    build.build()
    from denoising_sampler_step_gb300 import training
    return training


@pytest.fixture
def setup():
    g = torch.Generator(device="cuda").manual_seed(3)
    R, V = 12, 1003
    x = torch.zeros(R, 1004, device="cuda")
    x[:, :V] = 2 * torch.randn(R, V, generator=g, device="cuda")
    tok = torch.randint(V, (R,), generator=g, device="cuda").int()
    up = torch.randn(R, generator=g, device="cuda")
    mask = torch.rand(R, generator=g, device="cuda") > 0.3
    return g, x[:, :V], tok, up, mask


def grads(f, x):
    """The gradient of f at x, the logits in rows of 1,004 columns either way."""
    base = torch.zeros(x.shape[0], 1004, device="cuda", dtype=x.dtype)
    base[:, :1003] = x
    base.requires_grad_(True)
    f(base[:, :1003]).backward()
    return base.grad[:, :1003]


def same(a, b, scale):
    # both in fp32 on rows of 1,003 entries: some ten roundings of 2^-24 each of terms up to `scale`
    assert (a.double() - b.double()).abs().max() <= 2e-6 * scale


def test_token_logp_backward(T, setup):
    g, x, tok, up, mask = setup
    got = grads(lambda y: (up * T.token_logp(y, tok, 1.5, mask)).sum(), x)
    ref = grads(lambda y: (up * mask * torch.log_softmax(y / 1.5, 1).gather(1, tok[:, None].long())[:, 0]).sum(), x)
    same(got, ref, 4)
    assert not got[~mask].any()


@pytest.mark.parametrize("tail", [False, True])
def test_distill_backward(T, setup, tail):
    g, x, tok, up, mask = setup
    from denoising_sampler_step_gb300 import binding as B
    t = x + torch.randn(x.shape, generator=g, device="cuda")
    base = torch.zeros(12, 1004, device="cuda")
    base[:, :1003] = t
    top = B.dg_row_topk(base[:, :1003], 20, temperature=2.0, lse=True)
    lse = top["lse"] if tail else None
    got = grads(lambda y: (up * T.distill_loss(y, top["indices"], top["values"], lse, 2.0, mask)).sum(), x)

    def plain(y):
        logp = torch.log_softmax(y / 2, 1)
        idx = top["indices"].long()
        logq = top["values"] / 2 - (lse[:, None] if tail else (top["values"] / 2).logsumexp(1, keepdim=True))
        kl = (logq.exp() * (logq - logp.gather(1, idx))).sum(1)
        if tail:
            q0 = 1 - logq.exp().sum(1)
            kl = kl + q0 * (q0.log() - logp.scatter(1, idx, -float("inf")).logsumexp(1))
        return (4 * kl * up * mask).sum()
    same(got, grads(plain, x), 16)
    assert not got[~mask].any()


def test_policy_backward(T, setup):
    g, x, tok, up, mask = setup
    A, off = torch.randn(12, generator=g, device="cuda"), 0.5 * torch.randn(12, generator=g, device="cuda")
    logp0 = torch.log_softmax(x, 1).gather(1, tok[:, None].long())[:, 0]
    old, ref = logp0 + off, logp0 - 0.4
    got = grads(lambda y: (up * T.policy_loss(y, tok, old, A, ref, 0.2, 0.3, 0.1, mask=mask)[0]).sum(), x)

    def plain(y):
        logp = torch.log_softmax(y, 1).gather(1, tok[:, None].long())[:, 0]
        ratio = (logp - old).exp()
        loss = -torch.minimum(ratio * A, ratio.clamp(0.8, 1.3) * A) + 0.1 * ((ref - logp).exp() - 1 - (ref - logp))
        return (up * mask * loss).sum()
    same(got, grads(plain, x), 32)


def test_preference_backward_with_upstream_gradients(T, setup):
    g, x, tok, up, mask = setup
    start = torch.tensor([1, 4, 6, 6, 11], dtype=torch.int32, device="cuda")
    w = mask.float() * 0.5
    two = torch.tensor([0.7, -1.3], device="cuda")
    got = grads(lambda y: (two * T.preference_loss(y, tok, None, start, 0.3, 0.1, 1.0, w)[0]).sum(), x)

    def plain(y):
        logp = w * torch.log_softmax(y, 1).gather(1, tok[:, None].long())[:, 0]
        s = [logp[a:b].sum() for a, b in ((1, 4), (4, 6), (6, 6), (6, 11))]
        z = 0.3 * torch.stack([s[0] - s[1], s[2] - s[3]])
        return (two * (0.9 * torch.nn.functional.softplus(-z) + 0.1 * torch.nn.functional.softplus(z))).sum()
    same(got, grads(plain, x), 8)
    assert not got[0].any() and not got[11].any()


def test_the_training_run_improves_every_stage(T):
    from denoising_sampler_step_gb300 import finetune
    lines = []
    r = finetune.run(steps=40, log=lines.append)
    assert r["distill"][1] < 0.5 * r["distill"][0]
    assert r["policy"][1] > r["policy"][0] + 0.02
    assert r["preference"][1] > r["preference"][0] + 1.0
    assert len(lines) == 3 and np.isfinite([v for p in r.values() for v in p]).all()
