"""CPU oracle of the losses on the sampler's logits (fp64, plain and slow): the top logits of a
row, token log-probabilities, distillation from a teacher's top logits, the clipped policy loss
with a KL term and the preference loss, each with the gradient of the logits.

TEST INFRASTRUCTURE ONLY: the product path never calls it and shares no code with it.  Every
quantity is taken in float64 from its definition (include/dgsamp.h states them);
tests/test_loss_pins.py pins the gradients by central differences and the losses by closed
forms.  Rows of weight 0 (or with a negative token) give zeros and are not looked at.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def _logsumexp(z):
    m = np.max(z, axis=-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        return (m + np.log(np.sum(np.exp(z - m), axis=-1, keepdims=True)))[..., 0]


def row_topk(x, K: int, T: float = 1.0) -> dict:
    """The K largest entries per row, ties (and -0, +0) to the lowest index, and lse of x / T."""
    x = _f64(x)
    V = x.shape[1]
    idx = np.stack([np.lexsort((np.arange(V), -(row + 0.0)))[:K] for row in x]) if len(x) else np.zeros((0, K), int)
    return {"indices": idx.astype(np.int32), "values": np.take_along_axis(x, idx, 1), "lse": _logsumexp(x / T)}


def live_rows(R, weight=None, token=None):
    on = np.ones(R, bool) if weight is None else np.asarray(weight) != 0
    return on if token is None else on & (np.asarray(token) >= 0)


def token_logp(x, token, T: float = 1.0, weight=None) -> dict:
    R = len(x)
    on = live_rows(R, weight, token)
    logp, lse = np.zeros(R), np.zeros(R)
    z = _f64(x)[on] / T
    lse[on] = _logsumexp(z)
    logp[on] = z[np.arange(len(z)), np.asarray(token)[on]] - lse[on]
    return {"logp": logp, "lse": lse}


def token_grad(x, token, coef, T: float = 1.0, weight=None):
    """coef_r / T ([v == token] - p_v), coef = weight * dlogp."""
    g = np.zeros(np.shape(x))
    on = live_rows(len(g), weight, token)
    z = _f64(x)[on] / T
    d = -np.exp(z - _logsumexp(z)[:, None])
    d[np.arange(len(z)), np.asarray(token)[on]] += 1.0
    g[on] = d * (_f64(coef)[on] / T)[:, None]
    return g


def distill_loss(x, indices, teacher, teacher_lse=None, T: float = 1.0, weight=None) -> dict:
    R, V = np.shape(x)
    on = live_rows(R, weight)
    w = np.ones(R) if weight is None else _f64(weight)
    out = {"loss": np.zeros(R), "lse": np.zeros(R), "tail_logp": np.zeros(R), "grad": np.zeros((R, V))}
    for r in np.flatnonzero(on):
        z = _f64(x[r]) / T
        lse = _logsumexp(z)
        p = np.exp(z - lse)
        use = np.asarray(indices[r]) >= 0
        at, t = np.asarray(indices[r])[use], _f64(teacher[r])[use] / T
        inside = np.zeros(V, bool)
        inside[at] = True
        if teacher_lse is None:
            q = np.exp(t - _logsumexp(t)) if t.size and np.max(t) > -np.inf else np.zeros(t.size)
            q0 = 0.0
        else:
            q = np.exp(t - float(teacher_lse[r]))
            q0 = max(0.0, 1.0 - q.sum())
        pos = q > 0
        loss = np.sum(q[pos] * (np.log(q[pos]) - (z[at] - lse)[pos]))
        mass, share = q.sum(), 0.0
        if teacher_lse is not None:
            rest = z[~inside]
            logp0 = _logsumexp(rest) - lse if rest.size and np.max(rest) > -np.inf else -np.inf
            out["tail_logp"][r] = logp0
            # a bucket of masked entries (-inf, or the lowest value of fp32 or bf16) alone is left out
            if rest.size and np.max(rest) * T > -3.38e38 * min(T, 1.0):
                if logp0 < -87.0 and q0 <= (abs(float(teacher_lse[r])) + 4.0) * 2.0 ** -22:
                    q0 = 0.0       # what rounding leaves of 1 - sum q in fp32
                mass += q0
                share = np.zeros(V)
                share[~inside] = q0 * np.exp(rest - _logsumexp(rest))       # q_0 p_v / p_0
                if q0 > 0:
                    loss += q0 * (np.log(q0) - logp0)
        g = p * mass - share
        g[at] = mass * p[at] - q
        out["loss"][r], out["lse"][r], out["grad"][r] = T * T * loss, lse, w[r] * T * g
    return out


def policy_loss(x, token, old_logp, advantage, ref_logp=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                T: float = 1.0, weight=None) -> dict:
    R = len(x)
    on = live_rows(R, weight, token)
    w = np.ones(R) if weight is None else _f64(weight)
    o = token_logp(x, token, T, weight)
    logp, A = o["logp"], _f64(advantage)
    with np.errstate(over="ignore", invalid="ignore"):
        ratio = np.exp(logp - _f64(old_logp))
        raw, cut = ratio * A, np.clip(ratio, 1.0 - clip_low, 1.0 + clip_high) * A
        clipped = raw > cut
        loss, dlogp, kl = -np.minimum(raw, cut), np.where(clipped, 0.0, -raw), np.zeros(R)
        if ref_logp is not None:
            d = _f64(ref_logp) - logp
            kl = np.expm1(d) - d
            loss, dlogp = loss + kl_coef * kl, dlogp - kl_coef * np.expm1(d)
    for k, v in (("loss", loss), ("kl", kl), ("dlogp", dlogp)):
        o[k] = np.where(on, v, 0.0)
    o["clipped"] = (clipped & on).astype(np.uint8)
    o["grad"] = token_grad(x, token, w * o["dlogp"], T, weight)
    return o


def preference_loss(x, token, ref_logp, seq_start, beta=0.1, label_smoothing=0.0, T: float = 1.0, weight=None,
                    pair_weight=None) -> dict:
    R, P = len(x), len(seq_start) // 2
    on = live_rows(R, weight, token)
    w = np.where(on, 1.0 if weight is None else _f64(weight), 0.0)
    pw = np.ones(P) if pair_weight is None else _f64(pair_weight)
    o = token_logp(x, token, T, weight)
    term = w * np.where(on, o["logp"] - (0.0 if ref_logp is None else _f64(ref_logp)), 0.0)
    s = np.array([term[a:b].sum() for a, b in zip(seq_start[:-1], seq_start[1:])])
    z = beta * (s[0::2] - s[1::2])
    o["loss"] = (1 - label_smoothing) * np.logaddexp(0, -z) + label_smoothing * np.logaddexp(0, z)
    o["log_ratio"] = s
    dz = label_smoothing * np.exp(-np.logaddexp(0, -z)) - (1 - label_smoothing) * np.exp(-np.logaddexp(0, z))
    o["dlogp"] = np.zeros(R)
    for j in range(2 * P):
        sl = slice(seq_start[j], seq_start[j + 1])
        o["dlogp"][sl] = w[sl] * pw[j // 2] * beta * dz[j // 2] * (1 if j % 2 == 0 else -1)
    o["grad"] = token_grad(x, token, o["dlogp"], T, weight)
    return o
