"""The policy loss where a term's exponential leaves fp32's range and its coefficient is 0: the term is 0, as it is
in exact arithmetic."""
import numpy as np
import pytest
import torch

from oracle import loss_oracle as L
from test_gpu_losses import B, U, device_status_stays_clear, f32, i32, near, place, tol_logp  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1000, 100003])
def test_terms_of_coefficient_zero(B, dtype, V):
    rng = np.random.default_rng(V)
    x = rng.normal(0, 1, (4, V))
    x[:, 7] = 200.0                       # the token's ln p is about -200
    x, xf = place(x, dtype)
    tok = np.full(4, 11, np.int32)
    logp = L.token_logp(xf, tok)["logp"]
    tl = tol_logp(xf, tok, 1.0)
    close = (logp - 0.1).astype(np.float32)

    # the KL term reported, not trained on: e^195 - 1 - 195 is infinite in fp32
    ref = np.full(4, -5.0, np.float32)
    A = np.array([1.0, -0.5, 2.0, 0.0], np.float32)
    kw = dict(clip_low=0.2, clip_high=0.3, kl_coef=0.0)
    o = B.dg_policy_loss(x, i32(tok), f32(close), f32(A), ref_logp=f32(ref), grad=True, **kw)
    want = L.policy_loss(xf, tok, close, A, ref, **kw)
    assert (o["kl"] > 1e38).all()
    # |ratio A| below 2.3: derivative times the log-probability's error, a few roundings
    near(o["loss"], want["loss"], 2.3 * (tl + 16 * U), "loss")
    near(o["dlogp"], want["dlogp"], 2.3 * (tl + 16 * U), "dlogp")
    bare = B.dg_policy_loss(x, i32(tok), f32(close), f32(A), grad=True, **kw)
    assert torch.equal(o["grad"], bare["grad"]) and torch.equal(o["loss"], bare["loss"])

    # rows of advantage 0 (a group of equal rewards) under a ratio of e^100
    far = (logp - 100.0).astype(np.float32)
    kw["kl_coef"] = 0.1
    o = B.dg_policy_loss(x, i32(tok), f32(far), f32(np.zeros(4)), ref_logp=f32(close), grad=True, **kw)
    want = L.policy_loss(xf, tok, far, np.zeros(4), close, **kw)
    for k in ("loss", "dlogp", "kl"):
        near(o[k], want[k], 0.2 * (tl + 16 * U) if k != "kl" else tl + 16 * U, k)
    assert not o["clipped"].any() and torch.isfinite(o["grad"].float()).all()
