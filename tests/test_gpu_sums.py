"""The log-sum-exps at the accuracy of the kernels' own order of additions, and rows whose mass lies where one tile
or unit ends and the next begins.

Tolerances, from fp32 (u = 2^-24).  The losses' sums: a tile of at most 64 KB is folded by 256 threads or more in
groups of four vectors, so a thread adds 10 pairs and groups in a row at most (14 in bf16); then 5 steps in the
warp, 5 over the warps, tiles / 32 + 5 over a row's tiles.  A term carries the power of two's error, 4 u, and 3 u
of its exponent, on average over the row's distribution 3 u E with E = sum p (m - x) / T; a sum is rescaled at most
eight times, 6 u each.  m / T, ln s and their sum round once each.  In all

    TL = u (120 + tiles / 32 + 4 E + 2 (|m| / T + |lse|)).

The top logits' threads take every 2,048th group of 16 fp32 entries (or 4,096th of 32 bf16) of a row, one after the
other: V / 2,048 more, in place of the tiles.  An entry left out or counted twice at a boundary moves these rows'
log-sum-exp by at least 3e-3, some hundred times TL.
"""
import numpy as np
import pytest

from oracle import loss_oracle as L
from test_gpu_losses import B, U, device_status_stays_clear, f32, i32, near, place  # noqa: F401

pytestmark = pytest.mark.gpu

RING = 227 * 1024 - 4112


def tiling(V, dtype, K):
    """(entries of a tile, tiles) as in csrc/row_loss_plan.h."""
    N = 8 if dtype == "bf16" else 4
    nv = V // N
    if nv * 16 <= 64 * 1024:
        return max(V, 1), 1
    limit = (RING // (5 if K > 256 else 7) - 12 * K) // 128 * 8
    n = -(-nv // limit)
    per = (-(-nv // n) + 7) // 8 * 8
    return per * N, -(-nv // per)


def bound(xf, T, extra):
    z = xf / T
    m = z.max(1)
    lse = L._logsumexp(z)
    p = np.exp(z - lse[:, None])
    d = np.where(np.isfinite(z), m[:, None] - z, 0.0)
    return U * (120 + extra + 4 * (p * d).sum(1) + 2 * (np.abs(m) + np.abs(lse)))


def check(B, x, xf, T, K, dtype):
    R, V = xf.shape
    rng = np.random.default_rng(V)
    order = np.argsort(-xf, 1, kind="stable")
    tok = order[:, min(V - 1, 3)].astype(np.int32)
    z = xf / T
    want = L._logsumexp(z)
    ln_tok = z[np.arange(R), tok] - want
    rows = {}
    for k in (0, K):
        rows[k] = bound(xf, T, tiling(V, dtype, k)[1] / 32)
    one = f32(np.ones(R))
    for o in (B.dg_token_logp(x, i32(tok), temperature=T),
              B.dg_policy_loss(x, i32(tok), f32(ln_tok), one, temperature=T, grad=True)):
        near(o["lse"], want, rows[0], "lse")
        near(o["logp"], ln_tok, rows[0] + 4 * U * (np.abs(ln_tok) + 20), "logp")
    p = np.exp(z - want[:, None])
    g = -p
    g[np.arange(R), tok] += 1
    g *= o["dlogp"].double().cpu().numpy()[:, None] / T
    lnp = np.where(p > 0, -np.log(np.maximum(p, 1e-300)), 0.0)
    # (the ratio, about 1, is the kernel's own)
    tol = 2 / T * p * (rows[0][:, None] + U * (16 + 4 * lnp)) + 8 * U * np.abs(g)
    near(o["grad"], g, tol + 1e-37 + (2.0 ** -8 * np.abs(g) if dtype == "bf16" else 0), "gradient")

    # the teacher's entries: every other one of the largest, so that the bucket keeps boundary entries too
    n = min(V, 2 * K)
    idx = order[:, :n:2][:, :K].astype(np.int32)
    t = rng.normal(0, 1, idx.shape).astype(np.float32)
    inside = np.zeros(xf.shape, bool)
    np.put_along_axis(inside, idx, True, 1)
    rest = np.where(inside, -np.inf, z)
    tail = L._logsumexp(rest) - want
    tl_tail = rows[K] + bound(np.where(inside, -np.inf, xf), T, tiling(V, dtype, K)[1] / 32) + 4 * U * np.abs(tail)
    for grad in (False, True):
        o = B.dg_distill_loss(x, i32(idx), f32(t), f32(np.full(R, 9.0)), temperature=T, grad=grad)
        near(o["lse"], want, rows[K], "distillation's lse")
        near(o["tail_logp"], tail, tl_tail, "tail_logp")
    near(B.dg_row_topk(x, min(V, 5), temperature=T, lse=True)["lse"], want, bound(xf, T, V / 2048), "top logits' lse")


@pytest.mark.parametrize("V", [5, 1003, 16387, 32771, 50001, 100003, 262144, 1000003])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1.0, 1.3])
def test_spread_rows(B, V, dtype, T):
    rng = np.random.default_rng(V)
    x, xf = place(rng.normal(0, 1, (3, V)) * np.array([[0.1], [1.0], [4.0]]), dtype, 1)
    check(B, x, xf, T, min(V // 2, 64) or 1, dtype)


@pytest.mark.parametrize("V", [16387, 32771, 50001, 100003, 262144, 262151, 1000003])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [16, 300])
@pytest.mark.parametrize("low", [-60.0, -np.inf])
def test_mass_at_the_boundaries(B, V, dtype, K, low):
    """On either side of the losses' tiles (with and without lists) and of the top logits' units and tiles, and in the
    row's last entries, which no vector holds."""
    rng = np.random.default_rng(V + K)
    size = 2 if dtype == "bf16" else 4
    groups = [[e for e in range(step, V, step)] for step in (tiling(V, dtype, 0)[0], tiling(V, dtype, K)[0], 32768 // size)]
    groups.append([e for e in range(8192 // size, V, 8192 // size)])
    x = np.full((len(groups), V), low)
    for r, edges in enumerate(groups):
        if len(edges) > 40:
            edges = edges[:20] + edges[-20:]
        at = np.unique([0, V - 1, *range(V - V % (16 // size), V)] + [e - 1 for e in edges] + edges)
        x[r, at] = rng.uniform(-0.5, 0.5, len(at))
        if len(at) < 2 * K:      # the lists' other entries, of some mass of their own
            more = rng.permutation(V)[:3 * K]
            x[r, more] = np.where(x[r, more] == low, -8.0, x[r, more])
    x, xf = place(x, dtype, 1)
    check(B, x, xf, 1.0, K, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(B, dtype):
    """Rows that the top logits' CTAs share, and several rows per CTA of the losses'."""
    rng = np.random.default_rng(9)
    x, xf = place(rng.normal(0, 1, (310, 20011)) * rng.uniform(0.1, 4, (310, 1)), dtype)
    check(B, x, xf, 1.0, 40, dtype)
