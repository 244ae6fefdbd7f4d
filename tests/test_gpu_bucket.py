"""Distillation with a bucket in which the student has next to no probability, against the float64 oracle.

Tolerances, from fp32 (u = 2^-24): with D the largest distance of an entry from its group's maximum over T (the
teacher's entries and the bucket each have their own),

* TL = u (V / 64 + 80 + 4 D): ln of a group's sum, and a probability within the group (+ u (16 + 4 |ln|));
* ln p_0: the difference of two of those and of the maxima: 2 TL + 4 u |ln p_0|;
* q: EQ = u (8 (max|t| / T + |teacher_lse|) + K + 60), q_0 the same absolutely;
* loss / T^2: EQ (60 + |ln p_0|) + q_0 (2 TL + 4 u |ln p_0|) + 2 TL + 64 u;
* gradient in the bucket, w T e_v (M p_0 - q_0) with e_v the probability within it: its error times the
  coefficient, and EQ + p_0 (4 TL + 8 u) times e_v; on the entries, w T (M p_v - q_v): p_v and q_v likewise;
* from the saved lse and ln p_0, rounded once each: another 4 TL + 6 u (|lse| + |ln p_0|) of e_v and p_v;
* a bf16 gradient is rounded once: 2^-8 of itself on top.
"""
import numpy as np
import pytest

from oracle import loss_oracle as L
from test_gpu_losses import B, U, device_status_stays_clear, f32, i32, near, place  # noqa: F401

pytestmark = pytest.mark.gpu


def low_bucket(V, K, T, target, dtype, seed=0):
    """Three rows whose bucket has ln p_0 about `target`: equal entries, entries of unit spread, a third of them
    masked."""
    rng = np.random.default_rng(V + seed)
    x = rng.normal(0, 1, (3, V))
    x[0] = 0.0
    idx = np.stack([rng.permutation(V)[:K] for _ in range(3)]).astype(np.int32)
    idx[1, :2] = [0, V - 1]
    idx[1, 2:] = 2 + rng.permutation(V - 4)[:K - 2]
    top = rng.normal(0, 1, (3, K))
    x = x + T * (target - np.log(V - K)) - (0.5 if T == 1 else 0.0)
    x[2, rng.random(V) < 0.3] = -np.inf
    np.put_along_axis(x, idx, top, 1)
    t = (0.8 * top + rng.normal(0, 0.5, (3, K))).astype(np.float32)
    lse = (L._logsumexp(t.astype(np.float64) / T) + np.array([0.3, 0.5, 1.0])).astype(np.float32)
    return place(x, dtype, 1), idx, t, lse


def check(B, x, xf, idx, t, lse, T, w, dtype, K):
    V = xf.shape[1]
    kw = dict(teacher_lse=f32(lse), temperature=T)
    want = L.distill_loss(xf, idx, t, lse, T, w)
    inside = np.zeros(xf.shape, bool)
    np.put_along_axis(inside, idx, True, 1)
    z = xf / T
    zin, zout = np.where(inside, z, -np.inf), np.where(inside, -np.inf, z)
    below = lambda a: np.max(np.where(np.isfinite(a), a.max(1, keepdims=True) - a, 0))
    TL = U * (V / 64 + 80 + 4 * max(below(zin), below(zout)))
    far = np.abs(want["tail_logp"])
    EQ = U * (8 * (np.abs(t).max() / T + np.abs(lse).max()) + K + 60)
    q = np.where(inside, 0.0, 0.0)
    np.put_along_axis(q, idx, np.exp(t.astype(np.float64) / T - lse[:, None].astype(np.float64)), 1)
    q0 = 1 - q.sum(1)
    one = T * T * (EQ * (60 + far) + q0 * (2 * TL + 4 * U * far) + 2 * TL + 64 * U)

    def tol(extra):
        e = np.where(inside, 0.0, np.exp(zout - L._logsumexp(zout)[:, None]))
        p = np.where(inside, np.exp(zin - want["lse"][:, None]), 0.0)
        ln = lambda a: np.where(a > 0, -np.log(np.maximum(a, 1e-300)), 0.0)
        p0 = np.exp(want["tail_logp"])[:, None]
        coef = np.abs(p0 - q0[:, None])
        s = e * (coef * (TL + extra + U * (16 + 4 * ln(e))) + EQ + p0 * (4 * TL + 8 * U))
        s += p * (TL + extra + U * (16 + 4 * ln(p)) + EQ) + q * EQ
        s = np.abs(w)[:, None] * T * s + 8 * U * np.abs(want["grad"]) + 1e-37
        return s + (np.abs(want["grad"]) * 2.0 ** -8 if dtype == "bf16" else 0.0)

    o = B.dg_distill_loss(x, i32(idx), f32(t), weight=f32(w), grad=True, **kw)
    f = B.dg_distill_loss(x, i32(idx), f32(t), weight=f32(w), **kw)
    for a in (o, f):
        near(a["lse"], want["lse"], TL + 8 * U * (np.abs(want["lse"]) + 1), "lse")
        near(a["tail_logp"], want["tail_logp"], 2 * TL + 4 * U * far, "tail_logp")
        near(a["loss"], want["loss"], one, "loss")
    near(o["grad"], want["grad"], tol(0.0), "gradient")
    g = B.dg_distill_loss_backward(x, i32(idx), f32(t), o["lse"], f32(w), tail_logp=o["tail_logp"], **kw)
    near(g, want["grad"], tol(4 * TL + 6 * U * (np.abs(want["lse"]) + far).max()), "gradient from the saved values")


@pytest.mark.parametrize("V", [300, 4099, 100003, 262144])
@pytest.mark.parametrize("target", [-1.0, -60.0, -75.0, -80.0, -86.0, -88.0, -200.0, -5000.0])
@pytest.mark.parametrize("dtype,T", [("f32", 1.0), ("f32", 1.3), ("bf16", 1.0)])
@pytest.mark.parametrize("weight", [1.0, 65536.0])
def test_low_buckets(B, V, target, dtype, T, weight):
    """From 1 to 1e-2171, also where a loss scale multiplies the gradient."""
    (x, xf), idx, t, lse = low_bucket(V, 20, T, target, dtype)
    check(B, x, xf, idx, t, lse, T, np.full(3, weight), dtype, 20)


@pytest.mark.parametrize("V,K", [(16384, 1000), (262144, 700)])
def test_low_buckets_beside_long_lists(B, V, K):
    (x, xf), idx, t, lse = low_bucket(V, K, 1.0, -120.0, "f32")
    check(B, x, xf, idx, t, lse, 1.0, np.ones(3), "f32", K)


def test_rows_longer_than_the_chip(B):
    """The step in two passes: the second takes the bucket from what the first saved."""
    (x, xf), idx, t, lse = low_bucket(7000001, 20, 1.0, -120.0, "f32")
    check(B, x, xf, idx, t, lse, 1.0, np.ones(3), "f32", 20)


@pytest.mark.parametrize("target", [-50.0, -100.0, -1000.0])
def test_directional_differences(B, target):
    """(f(x + hu) - f(x - hu)) / 2h against the gradient, h = 2^-5: truncation h^2 / 6 of third derivatives below
    2 q_0, rounding 4 u |f| / 2h."""
    (x, xf), idx, t, lse = low_bucket(500, 20, 1.0, target, "f32")
    rng = np.random.default_rng(1)
    u = f32(rng.normal(0, 1, (3, 500)))
    h = 2.0 ** -5
    buf = lambda a: place(a.double().cpu().numpy(), "f32")[0]
    x[2][x[2] == -np.inf] = -2e4           # (differences of masked entries are none)
    f = lambda y, **k: B.dg_distill_loss(y, i32(idx), f32(t), f32(lse), **k)
    o = f(x, grad=True)
    g = (o["grad"] * u).sum(1).double().cpu().numpy()
    d = (f(buf(x + h * u))["loss"] - f(buf(x - h * u))["loss"]) / (2 * h)
    near(d, g, 1e-3 + 64 * U * np.abs(o["loss"].double().cpu().numpy()) * 4, "difference")
    assert (np.abs(g) > 1e-3).all()


@pytest.mark.parametrize("low", [-1e4, -1e9, -1e30, -3.4028235e38, -np.inf])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_mask_that_teacher_and_student_share(B, low, dtype):
    """The list holds all that is not masked: what fp32 leaves of 1 - sum q is no loss, however low the mask."""
    V, K = 4099, 30
    rng = np.random.default_rng(5)
    x = np.full((4, V), float(np.finfo(np.float32).min) if low == -3.4028235e38 and dtype == "f32" else
                -3.3895313892515355e38 if low == -3.4028235e38 else low)
    idx = np.stack([rng.permutation(V)[:K] for _ in range(4)]).astype(np.int32)
    np.put_along_axis(x, idx, rng.normal(0, 2, (4, K)) + 15, 1)
    x, xf = place(x, dtype)
    t = np.take_along_axis(xf, idx, 1).astype(np.float32)
    lse = L._logsumexp(t.astype(np.float64)).astype(np.float32)
    lse[3] = np.nextafter(lse[3], np.float32(np.inf))
    o = B.dg_distill_loss(x, i32(idx), f32(t), f32(lse), grad=True)
    # q = p but for roundings of lse (2 u |lse|) and q: first order in those
    EQ = U * (8 * (np.abs(t).max() + np.abs(lse).max()) + K + 60)
    near(o["loss"], np.zeros(4), 4 * EQ, "loss")
    near(o["grad"], np.zeros((4, V)), 4 * EQ, "gradient")
    g = B.dg_distill_loss_backward(x, i32(idx), f32(t), o["lse"], teacher_lse=f32(lse), tail_logp=o["tail_logp"])
    near(g, np.zeros((4, V)), 4 * EQ, "gradient from the saved values")


@pytest.mark.parametrize("target,kept", [(-80.0, True), (-86.0, True), (-88.0, False), (-100.0, False)])
def test_a_small_rest_counts_down_to_its_floor(B, target, kept):
    """q_0 = 15 u, which roundings of 1 - q could be: a term of the loss above ln p_0 = -87, also where every entry of
    the bucket is below fp32's range on its own, and none below."""
    V = 262144
    x = np.full((2, V), target - np.log(V - 1))
    x[0, 5] = x[1, V - 1] = 0.0
    x, xf = place(x, "f32")
    idx, t, lse = np.array([[5], [V - 1]], np.int32), np.full((2, 1), -15 * U, np.float32), np.zeros(2, np.float32)
    want = L.distill_loss(xf, idx, t, lse)
    assert (want["loss"] > 4e-5).all() if kept else (np.abs(want["loss"]) < 1e-5).all()
    # q_0 is off by the power of two's 4 u and two roundings, times |ln q_0 - ln p_0|
    tol = 6 * U * (14 + np.abs(target)) + 8 * U if kept else 30 * U
    o = B.dg_distill_loss(x, i32(idx), f32(t), f32(lse), grad=True)
    near(o["loss"], want["loss"], tol, "loss")
    g = B.dg_distill_loss_backward(x, i32(idx), f32(t), o["lse"], teacher_lse=f32(lse), tail_logp=o["tail_logp"])
    for v in (o["grad"], g):
        near(v.double().sum(1), np.zeros(2), 8 * U, "sum of the gradient")
        tail = v.double().clone()
        tail[[0, 1], idx[:, 0].tolist()] = 0
        near(tail.sum(1), [-15 * U if kept else 0.0] * 2, 7 * U if kept else U, "the bucket's gradient")
