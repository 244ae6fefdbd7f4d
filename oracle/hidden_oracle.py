"""CPU oracle, in float64, of the hidden stream's operators: embedding lookup and its gradient, RMS norm with
the residual's addition and its gradient, the tied 8-bit head.

TEST INFRASTRUCTURE ONLY: only the test suite may import this module; the product path never calls it and
shares no code with it.  Everything is taken from the definitions:

  out[r] = gamma W[token_r - s] for token_r in [s, e), else 0
  gW[v - s] = gamma sum over {r : token_r = v} of g[r]
  h = x + residual, rstd = (mean h^2 + eps)^(-1/2), y = h rstd w    (w: the weight with its offset)
  gradients of y's weighted sum by the chain rule, with rstd's dependence on h
  logits[r, v] = x_scale_r scale_v sum_k X[r, k] Q[v, k]
"""
from __future__ import annotations

import numpy as np


def token_embed(W, token, gamma: float, s: int = 0, e: int | None = None):
    """W: float64 rows of [s, e)."""
    e = s + W.shape[0] if e is None else e
    out = np.zeros((len(token), W.shape[1]))
    for r, t in enumerate(np.asarray(token, np.int64)):
        if s <= t < e:
            out[r] = gamma * W[t - s]
    return out


def token_embed_backward(g, token, gamma: float, s: int, e: int) -> dict:
    """grad [e - s, d]; size, the sum of the terms' magnitudes; count, the terms of each row."""
    d = g.shape[1]
    grad, size, count = np.zeros((e - s, d)), np.zeros((e - s, d)), np.zeros(e - s, np.int64)
    for r, t in enumerate(np.asarray(token, np.int64)):
        if s <= t < e:
            grad[t - s] += gamma * g[r]
            size[t - s] += np.abs(gamma * g[r])
            count[t - s] += 1
    return {"grad": grad, "size": size, "count": count}


def rms_norm(x, residual, w, eps: float) -> dict:
    h = x if residual is None else x + residual
    rstd = (np.mean(h * h, axis=1) + eps) ** -0.5
    return {"hidden": h, "rstd": rstd, "out": h * rstd[:, None] * w}


def rms_norm_backward(g, h, rstd, w, grad_hidden=None) -> dict:
    """For y_i = h_i rstd w_i: dy_i / dh_j = rstd w_i ([i = j] - rstd^2 h_i h_j / d)."""
    d = h.shape[1]
    inner = np.sum(g * w * h, axis=1)
    dh = rstd[:, None] * g * w - (rstd ** 3 * inner / d)[:, None] * h
    if grad_hidden is not None:
        dh = dh + grad_hidden
    return {"grad": dh, "grad_weight": np.sum(g * h * rstd[:, None], axis=0)}


def head(X, x_scale, W, scale):
    """X, W: float64 values of the codes."""
    return (X @ W.T) * np.asarray(x_scale, np.float64)[:, None] * np.asarray(scale, np.float64)[None, :]
