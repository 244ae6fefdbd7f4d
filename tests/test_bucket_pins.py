"""The distillation oracle's bucket of the entries outside the teacher's list, where the student has next to no
probability there: gradients by differences, and what is left out."""
import numpy as np
import pytest

from oracle import loss_oracle as L


def rows(gap, V=9):
    rng = np.random.default_rng(3)
    x = rng.normal(0, 1, (2, V))
    x[:, 4:] -= gap
    t = rng.normal(0, 1, (2, 4))
    lse = np.log(np.exp(t).sum(1)) + 0.7
    return x, np.tile(np.arange(4), (2, 1)), t, lse


@pytest.mark.parametrize("gap", [60.0, 86.0, 90.0, 200.0, 700.0, 5000.0])
def test_gradient_by_differences(gap):
    x, idx, t, lse = rows(gap)
    o = L.distill_loss(x, idx, t, lse)
    assert (o["tail_logp"] < -gap + 5).all() and (o["loss"] > 0.4 * gap).all()
    # the tail's gradient sums to -q_0 while p_0 is nothing beside it
    assert np.allclose(o["grad"][:, 4:].sum(1), np.exp(-0.7) - 1, atol=1e-8)
    h, g = 1e-4, np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (L.distill_loss(up, idx, t, lse)["loss"] - L.distill_loss(down, idx, t, lse)["loss"]).sum() / (2 * h)
    # truncation h^2 / 6, rounding 1e-16 of the loss over h
    assert np.abs(g - o["grad"]).max() < 1e-8 + 1e-11 * gap


def test_a_masked_bucket_is_left_out():
    x, idx, t, lse = rows(0.0)
    for low in (-np.inf, float(np.finfo(np.float32).min), -3.3895313892515355e38):
        x[:, 4:] = low
        o = L.distill_loss(x, idx, t, lse)
        q = np.exp(t - lse[:, None])
        p = np.exp(x[:, :4]) / np.exp(x[:, :4]).sum(1, keepdims=True)
        assert np.allclose(o["loss"], (q * np.log(q / p)).sum(1))
        assert np.allclose(o["grad"][:, :4], q.sum(1, keepdims=True) * p - q) and not o["grad"][:, 4:].any()


def test_a_rest_that_rounding_leaves_is_none():
    x, idx, t, lse = rows(1e4)
    lse = np.log(np.exp(t).sum(1)) + 1e-7
    assert (L.distill_loss(x, idx, t, lse)["loss"] < 10).all()
    assert (L.distill_loss(x + np.where(np.arange(9) >= 4, 9950, 0), idx, t, lse)["loss"] < 10).all()
    lse += 1e-3
    assert (L.distill_loss(x, idx, t, lse)["loss"] > 9).all()
