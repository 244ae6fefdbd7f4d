"""The losses on rows of logits and the top logits against the float64 oracle (oracle/loss_oracle.py).

Tolerances, derived from fp32 (u = 2^-24) before the kernels ran:

* lse, ln s: s is a sum of positive terms.  A thread adds at most V / 64 of them in a row (the
  narrowest launch), the merges a few more, each addition off by u: V u / 64 + 64 u.  A term's
  exponent (x - m) log2(e) / T is off by at most 3 u of itself, and |d| e^d <= 1/e; the exponential
  by 2^-22.  Adding m / T rounds by u |m / T|, as does the result: in all
  TOL = u (V / 64 + 80 + 4 max|z|).
* logp: TOL + 4 u (|z_token| + |lse|).
* a probability: relative TOL + u (16 + 4 |ln p|).
* what is computed from them carries these errors times its derivative, plus a few u of each term.
* a bf16 gradient is rounded once: 2^-8 of itself on top.
"""
import numpy as np
import pytest
import torch

from oracle import loss_oracle as L

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def B():
    from denoising_sampler_step_gb300 import build
    build.build()
    from denoising_sampler_step_gb300 import binding
    return binding


@pytest.fixture(autouse=True)
def device_status_stays_clear(B):
    yield
    B.dg_get_device_status()


def dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=dtype).cuda()


def f32(a):
    return dev(np.asarray(a, np.float32))


def i32(a):
    return dev(np.asarray(a, np.int32))


def logits(rng, R, V, dtype, pad=0, fill=float("nan"), scale=2.0):
    """(tensor [R, V] inside a wider buffer whose padding holds `fill`, its float64 values)."""
    x = rng.normal(0, 1, (R, V)) * rng.uniform(0.5, 2 * scale, (R, 1))
    return place(x, dtype, pad, fill)


def place(x, dtype, pad=0, fill=float("nan")):
    R, V = x.shape
    per = 16 // DT[dtype].itemsize
    ld = (V + per - 1) // per * per + pad * per
    buf = torch.full((R, ld), fill, dtype=DT[dtype], device="cuda")
    buf[:, :V] = torch.from_numpy(np.asarray(x, np.float32)).cuda()
    t = buf[:, :V]
    return t, t.double().cpu().numpy()


def tol_lse(x, T):
    z = np.abs(np.where(np.isfinite(x) & (np.abs(x) < 1e30), x, 0.0)) / T
    return U * (x.shape[1] / 64 + 80 + 4 * z.max())


def tol_logp(x, token, T):
    z = x[np.arange(len(x)), np.maximum(token, 0)] / T
    z = np.where(np.isfinite(z), z, 0.0)
    return tol_lse(x, T) + 4 * U * (np.abs(z) + np.abs(z).max() + 30)


def near(got, want, tol, what):
    got, want = got.detach().double().cpu().numpy(), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        off = np.where(same, 0.0, np.abs(got - want))
    worst = np.max(off - np.broadcast_to(tol, off.shape), initial=-np.inf)
    assert not np.isnan(worst) and worst <= 0, f"{what}: {worst} over the tolerance, off by {np.nanmax(off)}"


def grad_tol(want, p, coef, x, T, dtype, rel_coef=0.0):
    """Of g = coef (hot - p) style gradients: the probability's error times the coefficient, the
    coefficient's own relative error, a few roundings, and the storage type's."""
    with np.errstate(divide="ignore"):
        lnp = np.where(p > 0, -np.log(np.maximum(p, 1e-300)), 0.0)
    rel_p = tol_lse(x, T) + U * (16 + 4 * lnp)
    tol = np.abs(coef)[:, None] * (p * rel_p + 4 * U * np.abs(p)) + np.abs(want) * (rel_coef + 8 * U) + 1e-37
    return tol + (np.abs(want) * 2.0 ** -8 if dtype == "bf16" else 0.0)


def softmax(x, T):
    z = x / T
    return np.exp(z - L._logsumexp(z)[:, None])


def mask_of(rng, R, share=0.3):
    w = rng.uniform(0.2, 2.0, R).astype(np.float32)
    w[rng.random(R) < share] = 0.0
    return w


# vocabularies: one to a few entries, around vectors of 4 and 8, around chunks, odd ones, the full one
VOCABS = [1, 2, 3, 4, 7, 9, 31, 257, 1000, 4095, 4096, 4099, 8191, 8193, 16384, 32003, 100003, 262144]
# rows of a wide and of a narrow call
CASES = [(3, V, "f32") for V in VOCABS] + [(3, V, "bf16") for V in VOCABS] + \
        [(1, 262144, "f32"), (1, 5, "bf16"), (700, 33, "f32"), (611, 1025, "bf16"), (40, 65537, "f32"),
         (90, 50001, "bf16"), (3, 500009, "f32"), (2, 1000003, "bf16"), (2, 2500001, "f32")]


# --------------------------------------------------------------------------- tokens and the policy loss

def token_case(R, V, dtype, seed=0, pad=0):
    rng = np.random.default_rng(1000 * R + V + seed)
    x, xf = logits(rng, R, V, dtype, pad)
    tok = rng.integers(0, V, R).astype(np.int32)
    tok[0] = V - 1
    return rng, x, xf, tok


@pytest.mark.parametrize("R,V,dtype", CASES)
@pytest.mark.parametrize("T", [1.0, 1.3])
def test_token_logp_and_its_gradient(B, R, V, dtype, T):
    rng, x, xf, tok = token_case(R, V, dtype, pad=R % 2)
    w = mask_of(rng, R)
    w[0] = 1.0
    if R > 2:
        tok[R - 1] = -1
    o = B.dg_token_logp(x, i32(tok), temperature=T, weight=f32(w))
    want = L.token_logp(xf, tok, T, w)
    near(o["lse"], want["lse"], tol_lse(xf, T), "lse")
    near(o["logp"], want["logp"], tol_logp(xf, tok, T), "logp")

    d = rng.normal(0, 1, R).astype(np.float32)
    out = place(np.full((R, V), 7.0), dtype, 1, fill=5.0)[0]
    g = B.dg_token_logp_backward(x, i32(tok), o["lse"], f32(d), scale=f32(w), temperature=T, out=out)
    want_g = L.token_grad(xf, tok, w.astype(np.float64) * d, T, w)
    near(g, want_g, grad_tol(want_g, softmax(xf, T), w * d / T, xf, T, dtype, 4 * U), "gradient")
    assert (out._base[:, V:] == 5.0).all(), "the padding was written"


@pytest.mark.parametrize("R,V,dtype", CASES)
@pytest.mark.parametrize("T,kl_coef", [(1.0, 0.04), (0.7, 0.0)])
def test_policy_loss(B, R, V, dtype, T, kl_coef):
    rng, x, xf, tok = token_case(R, V, dtype, 1, pad=1)
    w = mask_of(rng, R)
    w[0] = 1.0
    logp = L.token_logp(xf, tok, T)["logp"]
    ratio = rng.uniform(0.5, 1.6, R)
    for edge in (0.8, 1.3):
        ratio = np.where(np.abs(ratio - edge) < 5e-3, edge + 1e-2, ratio)
    old = (logp - np.log(ratio)).astype(np.float32)
    ref = (logp + rng.normal(0, 0.3, R)).astype(np.float32) if kl_coef else None
    A = rng.normal(0, 1, R).astype(np.float32)
    kw = dict(clip_low=0.2, clip_high=0.3, kl_coef=kl_coef)
    o = B.dg_policy_loss(x, i32(tok), f32(old), f32(A), ref_logp=None if ref is None else f32(ref), temperature=T,
                         weight=f32(w), grad=True, **kw)
    want = L.policy_loss(xf, tok, old, A, ref, T=T, weight=w, **kw)
    near(o["lse"], want["lse"], tol_lse(xf, T), "lse")
    tl = tol_logp(xf, tok, T)
    near(o["logp"], want["logp"], tl, "logp")
    assert np.array_equal(o["clipped"].cpu().numpy(), want["clipped"])
    # exp(d) and exp(logp - old) stay below 2 and 4: derivative times tl, a few roundings of each term
    size = 2 * np.abs(A) + 4 * kl_coef + 1e-30
    near(o["kl"], want["kl"], 4 * tl + 16 * U, "kl")
    near(o["loss"], want["loss"], size * (tl + 16 * U), "loss")
    near(o["dlogp"], want["dlogp"], size * (tl + 16 * U), "dlogp")
    # the gradient is linear in dlogp: the kernel's own dlogp isolates the rest
    mine = o["dlogp"].double().cpu().numpy()
    want_g = L.token_grad(xf, tok, w.astype(np.float64) * mine, T, w)
    near(o["grad"], want_g, grad_tol(want_g, softmax(xf, T), w * mine / T, xf, T, dtype, 4 * U), "gradient")

    f = B.dg_policy_loss(x, i32(tok), f32(old), f32(A), ref_logp=None if ref is None else f32(ref), temperature=T,
                         weight=f32(w), **kw)
    for k in ("loss", "logp", "lse", "kl", "dlogp", "clipped"):
        # another order of additions at most
        near(f[k], o[k].double().cpu().numpy(), size * (2 * tl + 32 * U) if k != "lse" else 2 * tol_lse(xf, T), k)


# --------------------------------------------------------------------------- distillation

def distill_case(R, V, K, dtype, T, tail, seed=0, pad=0):
    rng = np.random.default_rng(7000 * R + V + K + seed)
    x, xf = logits(rng, R, V, dtype, pad)
    teacher = (0.8 * xf + rng.normal(0, 1.0, (R, V))).astype(np.float32)
    idx = np.argpartition(-teacher, min(K, V) - 1, 1)[:, :K].astype(np.int32)
    t = np.take_along_axis(teacher, idx, 1)
    lse = L._logsumexp(teacher.astype(np.float64) / T).astype(np.float32) if tail else None
    return rng, x, xf, idx, t, lse


def check_distill(B, x, xf, idx, t, lse, T, w, dtype, backward=True):
    K = idx.shape[1]
    kw = dict(teacher_lse=None if lse is None else f32(lse), temperature=T)
    o = B.dg_distill_loss(x, i32(idx), f32(t), weight=None if w is None else f32(w), grad=True, **kw)
    want = L.distill_loss(xf, idx, t, lse, T, w)
    tl = tol_lse(xf, T)
    near(o["lse"], want["lse"], tl, "lse")
    near(o["tail_logp"], want["tail_logp"], 2 * tl + 8 * U * 40, "tail_logp") if lse is not None else None
    # q_k: relative error 4 u (|t_k| + |off|) / T + (K + 40) u, the sum q_0 the same absolutely; ln q - ln p
    # adds tl and 4 u |z|; everything stays below 60 nats
    zmax = np.abs(np.where(np.abs(xf) < 1e30, xf, 0)).max() / T + np.abs(t[np.abs(t) < 1e30]).max(initial=0) / T
    eq = U * (8 * zmax + K + 60)
    one = T * T * (60 * eq + 2 * tl + 8 * U * zmax + 64 * U)
    near(o["loss"], want["loss"], one, "loss")
    p = softmax(xf, T)
    ww = np.ones(len(xf)) if w is None else w.astype(np.float64)
    # p M and q carry tl + eq; a tail entry p (M - q_0 / p_0): eq / p_0 + 2 tl q_0 / p_0 as well
    tol = grad_tol(want["grad"], p, ww * T, xf, T, dtype, 0.0)
    tol += (np.abs(ww) * T)[:, None] * p * (2 * eq + 2 * tl)
    if lse is not None:
        p0 = np.exp(want["tail_logp"])[:, None]
        tol += (np.abs(ww) * T)[:, None] * p * np.minimum(1.0 / p0, 1e9) * (2 * eq + 4 * tl + 400 * U)
    q = np.zeros_like(p)
    for r in range(len(xf)):
        use = idx[r] >= 0
        tt = t[r][use].astype(np.float64) / T
        if tt.size and tt.max() > -np.inf:
            q[r, idx[r][use]] = np.exp(tt - (L._logsumexp(tt) if lse is None else lse[r]))
    tol += (np.abs(ww) * T)[:, None] * q * eq
    near(o["grad"], want["grad"], tol, "gradient")
    if backward:
        g = B.dg_distill_loss_backward(x, i32(idx), f32(t), o["lse"], None if w is None else f32(w),
                                       tail_logp=o.get("tail_logp"), **kw)
        near(g, want["grad"], 2 * tol, "gradient from the saved values")
        f = B.dg_distill_loss(x, i32(idx), f32(t), weight=None if w is None else f32(w), **kw)
        near(f["loss"], want["loss"], one, "loss alone")
        near(f["lse"], want["lse"], tl, "lse alone")
    return o, want


@pytest.mark.parametrize("R,V,dtype", CASES)
@pytest.mark.parametrize("T,tail", [(1.0, False), (1.4, True)])
def test_distill_loss(B, R, V, dtype, T, tail):
    K = min(V, {1: 1, 0: 5, 2: 64}[V % 3])
    rng, x, xf, idx, t, lse = distill_case(R, V, K, dtype, T, tail, pad=R % 2)
    w = mask_of(rng, R)
    w[0] = 1.0
    check_distill(B, x, xf, idx, t, lse, T, w, dtype)


@pytest.mark.parametrize("K", [1, 2, 31, 33, 200, 512, 1024])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_entry_counts(B, K, tail, dtype):
    rng, x, xf, idx, t, lse = distill_case(5, 9001, K, dtype, 1.0, tail)
    idx[1, ::2] = -1          # padded entries
    idx[2] = -1               # a row without entries: loss and gradient 0
    t[3, K // 2:] = -np.inf   # the teacher rules some of its entries out
    o, _ = check_distill(B, x, xf, idx, t, lse, 1.0, None, dtype)
    assert float(o["loss"][2]) == 0.0 and not o["grad"][2].any()


def test_distill_over_the_whole_vocabulary(B):
    """K = V: the bucket is empty, its term is left out."""
    rng, x, xf, idx, t, lse = distill_case(4, 37, 37, "f32", 1.0, True)
    want = L.distill_loss(xf, idx, t, None)
    o = B.dg_distill_loss(x, i32(idx), f32(t), teacher_lse=f32(lse), grad=True)
    # q sums to 1 within 40 u of the full softmax: first order terms below 60 nats
    near(o["loss"], want["loss"], 1e-5, "loss")
    near(o["grad"], want["grad"], 2e-6, "gradient")
    assert (o["tail_logp"] == -float("inf")).all()


def test_distill_entries_at_the_edges(B):
    """Entries at the first and last columns, beside slice and chunk borders, and all in one place."""
    for V, dtype in ((262144, "f32"), (262144, "bf16"), (131075, "f32"), (500009, "f32")):
        rng, x, xf, idx, t, lse = distill_case(3, V, 64, dtype, 1.0, True, seed=5)
        idx[0, :8] = [0, V - 1, 1, V - 2, 2, V - 3, 3, V - 4]
        idx[0, 8:] = V // 2 + np.arange(56)
        idx[1] = V - 64 + np.arange(64)
        idx[2] = np.arange(64)[::-1]
        lse = lse + 3.0       # most of the teacher's mass lies in the bucket
        check_distill(B, x, xf, idx, t, lse, 1.0, None, dtype)


# --------------------------------------------------------------------------- preference

@pytest.mark.parametrize("V,dtype", [(33, "f32"), (4099, "bf16"), (32003, "bf16"), (262144, "f32")])
@pytest.mark.parametrize("smoothing,ref_free", [(0.0, False), (0.1, True)])
def test_preference_loss(B, V, dtype, smoothing, ref_free):
    rng = np.random.default_rng(V + ref_free)
    lens = [3, 0, 1, 5, 7, 2, 0, 0]
    start = np.concatenate([[2], 2 + np.cumsum(lens)])    # rows 0, 1 and the last two in no sequence
    R, n = int(start[-1]) + 2, len(lens) // 2
    x, xf = logits(rng, R, V, dtype, 1)
    tok = rng.integers(0, V, R).astype(np.int32)
    tok[5] = -1
    w = mask_of(rng, R, 0.2)
    w[0] = 1.0
    pw = np.array([1.0, 0.5, 0.0, 2.0], np.float32)
    logp = L.token_logp(xf, np.maximum(tok, 0), 1.2)["logp"]
    ref = None if ref_free else (logp + rng.normal(0, 0.5, R)).astype(np.float32)
    kw = dict(beta=0.3, label_smoothing=smoothing, temperature=1.2)
    args = (i32(tok), None if ref is None else f32(ref), i32(start))
    o = B.dg_preference_loss(x, *args, weight=f32(w), pair_weight=f32(pw), grad=True, **kw)
    kw["T"] = kw.pop("temperature")
    want = L.preference_loss(xf, tok, ref, start, weight=w, pair_weight=pw, **kw)
    tl = tol_logp(xf, tok, 1.2)
    near(o["logp"], want["logp"], tl, "logp")
    near(o["lse"], want["lse"], tol_lse(xf, 1.2), "lse")
    ts = np.array([(np.abs(w) * (tl + 4 * U * 20))[a:b].sum() for a, b in zip(start[:-1], start[1:])])
    near(o["log_ratio"], want["log_ratio"], ts + U * np.abs(want["log_ratio"]) + 1e-30, "log_ratio")
    tz = 0.3 * (ts[0::2] + ts[1::2])
    near(o["loss"], want["loss"], tz + 8 * U * (1 + want["loss"]), "loss")
    td = np.zeros(R)
    for j in range(2 * n):
        td[start[j]:start[j + 1]] = 0.3 * pw[j // 2] * (tz[j // 2] + 16 * U)
    near(o["dlogp"], want["dlogp"], td * np.abs(w) + 1e-30, "dlogp")
    mine = o["dlogp"].double().cpu().numpy()
    assert not mine[:2].any() and not mine[-2:].any() and not mine[5]
    want_g = L.token_grad(xf, tok, mine, 1.2, w)
    near(o["grad"], want_g, grad_tol(want_g, softmax(xf, 1.2), mine / 1.2, xf, 1.2, dtype, 4 * U), "gradient")
    g = B.dg_token_logp_backward(x, args[0], o["lse"], o["dlogp"], temperature=1.2)
    near(g, want_g, grad_tol(want_g, softmax(xf, 1.2), mine / 1.2, xf, 1.2, dtype, 4 * U), "backward call")


def test_preference_many_pairs_and_long_sequences(B):
    rng = np.random.default_rng(3)
    lens = np.concatenate([[900, 1100], rng.integers(0, 4, 400)])
    start = np.concatenate([[0], np.cumsum(lens)])
    R = int(start[-1])
    x, xf = logits(rng, R, 100, "f32")
    tok = rng.integers(0, 100, R).astype(np.int32)
    logp = L.token_logp(xf, tok)["logp"]
    ref = (logp + rng.normal(0, 0.2, R)).astype(np.float32)
    o = B.dg_preference_loss(x, i32(tok), f32(ref), i32(start), beta=0.05, grad=True)
    want = L.preference_loss(xf, tok, ref, start, beta=0.05)
    tl = tol_logp(xf, tok, 1.0) + 80 * U
    ts = np.array([tl[a:b].sum() for a, b in zip(start[:-1], start[1:])])
    near(o["log_ratio"], want["log_ratio"], ts + U * np.abs(want["log_ratio"]) + 1e-30, "log_ratio")
    near(o["loss"], want["loss"], 0.05 * (ts[0::2] + ts[1::2]) + 8 * U * (1 + want["loss"]), "loss")


def test_preference_without_rows(B):
    x = torch.empty((0, 8), device="cuda")
    none = torch.empty(0, device="cuda")
    o = B.dg_preference_loss(x, none.int(), none, i32([0, 0, 0]), grad=True)
    near(o["loss"], [np.log(2.0)], 4 * U, "loss")


# --------------------------------------------------------------------------- masks and extremes

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [64, 4099, 262144])
def test_rows_left_out_are_not_looked_at(B, dtype, V):
    rng = np.random.default_rng(V)
    x, xf = logits(rng, 6, V, dtype, 1)
    w = np.array([1, 0, 0, 1, 0, 1], np.float32)
    tok = np.array([1, 2, 3, -1, 5, 6], np.int32)
    x[1], x[2, ::2], x[4, 1::3] = float("nan"), float("inf"), -float("inf")
    x[3] = float("nan")    # left out by its token
    idx = np.tile(np.arange(8, dtype=np.int32), (6, 1))
    t = f32(rng.normal(0, 1, (6, 8)))
    ones, nan = f32(np.ones(6)), f32(np.full(6, np.nan))
    old = torch.where(f32(w) != 0, -ones, nan)
    pol = B.dg_policy_loss(x, i32(tok), old, ones, ref_logp=old, kl_coef=0.1, weight=f32(w), grad=True)
    lp = B.dg_token_logp(x, i32(tok), weight=f32(w))
    bwd = {"grad": B.dg_token_logp_backward(x, i32(tok), lp["lse"], ones, scale=f32(w))}
    pref = B.dg_preference_loss(x, i32(tok), old, i32([0, 3, 6]), weight=f32(w), grad=True)
    for o in (pol, lp, bwd, pref):
        for k, v in o.items():
            assert torch.isfinite(v.float()).all(), k
            if v.shape[0] == 6 and k != "log_ratio":
                for r in (1, 2, 3, 4):
                    assert not v[r].any(), (k, r)
    w[3] = 0
    o = B.dg_distill_loss(x, i32(idx), t, teacher_lse=4 * ones, weight=f32(w), grad=True)
    g = B.dg_distill_loss_backward(x, i32(idx), t, o["lse"], f32(w), teacher_lse=4 * ones, tail_logp=o["tail_logp"])
    for v in (*o.values(), g):
        assert torch.isfinite(v.float()).all() and not v[1:3].any() and not v[4].any() and v[0].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("low", [-np.inf, float(np.finfo(np.float32).min)])
@pytest.mark.parametrize("V", [100, 32003, 262144])
def test_masked_vocabulary(B, dtype, low, V):
    """Most entries masked by -inf or by the type's lowest value: probability and gradient 0."""
    rng = np.random.default_rng(V)
    if dtype == "bf16" and np.isfinite(low):
        low = float(torch.finfo(torch.bfloat16).min)
    x, xf = logits(rng, 4, V, dtype)
    keep = np.zeros((4, V), bool)
    keep[:, rng.permutation(V)[:20]] = True
    keep[1] = False
    keep[1, V - 1] = True      # one entry left: one-hot
    xf = np.where(keep, xf, low)
    x, xf = place(xf, dtype)
    tok = np.array([np.flatnonzero(k)[-1] for k in keep], np.int32)
    A = f32([1, -1, 2, 0.5])
    old = f32(L.token_logp(xf, tok)["logp"])
    o = B.dg_policy_loss(x, i32(tok), old, A, grad=True)
    want = L.policy_loss(xf, tok, old.cpu().numpy(), A.cpu().numpy())
    tl = tol_logp(xf, tok, 1.0)
    near(o["logp"], want["logp"], tl, "logp")
    mine = o["dlogp"].double().cpu().numpy()
    want_g = L.token_grad(xf, tok, mine)
    near(o["grad"], want_g, grad_tol(want_g, softmax(xf, 1.0), mine, xf, 1.0, dtype), "gradient")
    idx = np.stack([np.flatnonzero(k)[np.arange(4) % k.sum()] for k in keep]).astype(np.int32)
    idx[1, 1:] = -1
    idx[2, 3] = np.flatnonzero(~keep[2])[0]     # the teacher's entry is masked for the student,
    t = rng.normal(0, 1, (4, 4)).astype(np.float32)
    t[2, 3] = -np.inf                           # and has no mass
    for lse in (None, f32([3, 3, 3, 3])):
        check_distill(B, x, xf, idx, t, None if lse is None else lse.cpu().numpy(), 1.0, None, dtype)


def test_a_masked_token_and_a_masked_teacher_entry(B):
    x = torch.zeros((2, 64), device="cuda")
    x[:, 10] = -float("inf")
    o = B.dg_policy_loss(x, i32([10, 11]), f32([-4, -4]), f32([1, 1]), grad=True)
    assert float(o["logp"][0]) == -float("inf") and float(o["loss"][0]) == 0.0 and not o["grad"][0].any()
    t = f32([[1, 1], [1, 1]])
    o = B.dg_distill_loss(x, i32([[10, 11], [12, 13]]), t, grad=True)
    assert float(o["loss"][0]) == float("inf")
    near(o["grad"][0, 10], -0.5, 4 * U, "gradient at the impossible entry")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [3, 4097, 262144])
def test_a_row_without_a_distribution_gives_nan(B, dtype, V):
    x, _ = place(np.full((2, V), -np.inf), dtype)
    x[1] = 0.5
    o = B.dg_token_logp(x, i32([0, 1]))
    assert torch.isnan(o["lse"][0]) and torch.isnan(o["logp"][0])
    near(o["lse"][1:], [0.5 + np.log(V)], U * (V / 64 + 100), "lse of a constant row")
    p = B.dg_policy_loss(x, i32([0, 1]), f32([-1, -1]), f32([1, 1]), grad=True)
    assert torch.isnan(p["grad"][0].float()).all() and torch.isfinite(p["grad"][1].float()).all()
    d = B.dg_distill_loss(x, i32([[0], [1]]), f32([[1], [1]]), grad=True)
    assert torch.isnan(d["loss"][0]) and torch.isfinite(d["grad"][1].float()).all()
    k = B.dg_row_topk(x, 3, lse=True)
    assert torch.isnan(k["lse"][0]) and k["indices"].tolist() == [[0, 1, 2], [0, 1, 2]]


def test_rows_longer_than_the_chip(B):
    """More tiles than all SMs' shared memory holds: the row is read a second time for its gradient."""
    R, V, K = 2, 7000001, 40
    rng, x, xf, tok = token_case(R, V, "f32", pad=1)
    logp = L.token_logp(xf, tok, 1.0)["logp"]
    old, A = (logp - 0.1).astype(np.float32), np.float32([0.5, -1.5])
    o = B.dg_policy_loss(x, i32(tok), f32(old), f32(A), grad=True)
    want = L.policy_loss(xf, tok, old, A, None, T=1.0, weight=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0)
    tl = tol_logp(xf, tok, 1.0)
    near(o["loss"], want["loss"], 2 * np.abs(A) * (tl + 16 * U), "loss")
    mine = o["dlogp"].double().cpu().numpy()
    want_g = L.token_grad(xf, tok, mine, 1.0, None)
    near(o["grad"], want_g, grad_tol(want_g, softmax(xf, 1.0), mine, xf, 1.0, "f32", 4 * U), "gradient")
    rng, x, xf, idx, t, lse = distill_case(R, V, K, "f32", 1.4, True)
    check_distill(B, x, xf, idx, t, lse, 1.4, np.float32([1.0, 0.5]), "f32")


@pytest.mark.parametrize("gap", [50.0, 1e4, 1e30])
def test_one_hot_rows(B, gap):
    xf = np.zeros((2, 5000))
    xf[0, 4321] = gap
    xf[1, 17] = -gap
    x, xf = place(xf, "f32")
    tok = np.array([4321, 17], np.int32)
    o = B.dg_policy_loss(x, i32(tok), f32([0, 0]), f32([1, 1]), grad=True)
    want = L.token_logp(xf, tok)
    near(o["logp"], want["logp"], U * (300 + 8 * np.abs(want["logp"])), "logp")
    assert torch.isfinite(o["grad"]).all()


def test_offsets_past_32_bits(B):
    """Rows further apart than 2^31 elements: logits and gradients (12 GB of address range each)."""
    ld, V = (1 << 30) + 4, 4099
    buf = torch.empty(2 * ld + 8192, device="cuda")
    gbuf = torch.empty(2 * ld + 8192, device="cuda")
    x, g = (b.as_strided((3, V), (ld, 1)) for b in (buf, gbuf))
    rng = np.random.default_rng(0)
    x.copy_(torch.from_numpy(rng.normal(0, 2, (3, V)).astype(np.float32)))
    xf = x.double().cpu().numpy()
    tok = np.array([0, 5, V - 1], np.int32)
    out = {"grad": g}
    B.dg_policy_loss(x, i32(tok), f32([-5, -5, -5]), f32([1, 1, 1]), out=out)
    mine = out["dlogp"].double().cpu().numpy()
    want_g = L.token_grad(xf, tok, mine)
    near(g, want_g, grad_tol(want_g, softmax(xf, 1.0), mine, xf, 1.0, "f32"), "gradient")
    top = B.dg_row_topk(x, 7)
    assert np.array_equal(top["indices"].cpu().numpy(), L.row_topk(xf, 7)["indices"])
    o = B.dg_distill_loss(x, top["indices"], top["values"], out={"grad": g})
    want = L.distill_loss(xf, *(top[k].cpu().numpy() for k in ("indices", "values")))
    near(o["loss"], want["loss"], 1e-4, "loss")


# --------------------------------------------------------------------------- memory, streams, graphs, repeats

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,V", [(5, 4099), (40, 262144), (300, 1000)])
def test_the_gradient_may_replace_the_logits(B, dtype, R, V):
    rng, x, xf, idx, t, lse = distill_case(R, V, 16, dtype, 1.0, True)
    tok, w = i32(rng.integers(0, V, R)), f32(mask_of(rng, R))
    A, old = f32(rng.normal(0, 1, R)), f32(np.full(R, -9.0))
    apart = B.dg_policy_loss(x, tok, old, A, weight=w, grad=True)
    y = torch.empty_like(x._base).copy_(x._base)[:, :V]
    B.dg_policy_loss(y, tok, old, A, weight=w, out={"grad": y})
    assert torch.equal(y, apart["grad"])
    apart = B.dg_distill_loss(x, i32(idx), f32(t), f32(lse), weight=w, grad=True)
    y = torch.empty_like(x._base).copy_(x._base)[:, :V]
    B.dg_distill_loss(y, i32(idx), f32(t), f32(lse), weight=w, out={"grad": y})
    assert torch.equal(y, apart["grad"])
    apart_b = B.dg_distill_loss_backward(x, i32(idx), f32(t), apart["lse"], w, f32(lse), apart["tail_logp"])
    y = torch.empty_like(x._base).copy_(x._base)[:, :V]
    B.dg_distill_loss_backward(y, i32(idx), f32(t), apart["lse"], w, f32(lse), apart["tail_logp"], out=y)
    assert torch.equal(y, apart_b)


@pytest.mark.parametrize("V", [1000, 100003, 262144])
def test_calls_repeat_bit_for_bit(B, V):
    rng, x, xf, idx, t, lse = distill_case(70, V, 50, "f32", 1.0, True)
    tok, one = i32(rng.integers(0, V, 70)), f32(np.ones(70))
    runs = [(B.dg_policy_loss(x, tok, -9 * one, one, grad=True), B.dg_distill_loss(x, i32(idx), f32(t), f32(lse), grad=True),
             B.dg_row_topk(x, 50, lse=True), B.dg_preference_loss(x, tok, None, i32([0, 30, 70]), grad=True))
            for _ in range(3)]
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            for k in a:
                assert torch.equal(a[k], b[k]), k


def test_calls_run_on_the_given_stream_and_in_a_graph(B):
    rng, x, xf, idx, t, lse = distill_case(20, 30011, 40, "bf16", 1.0, False)
    s = torch.cuda.Stream()
    y = torch.zeros_like(x._base)
    src = x._base.clone()
    s.wait_stream(torch.cuda.current_stream())
    ii, tt, tok, one = i32(idx), f32(t), i32(np.arange(20)), f32(np.ones(20))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)      # the inputs arrive late on the side stream
        y.copy_(src)
    d = B.dg_distill_loss(y[:, :30011], ii, tt, grad=True, stream=s)
    k = B.dg_row_topk(y[:, :30011], 40, lse=True, stream=s)
    p = B.dg_preference_loss(y[:, :30011], tok, None, i32([0, 9, 20]), grad=True, stream=s)
    s.synchronize()
    want = (B.dg_distill_loss(x, ii, tt, grad=True), B.dg_row_topk(x, 40, lse=True),
            B.dg_preference_loss(x, tok, None, i32([0, 9, 20]), grad=True))
    for a, b in zip((d, k, p), want):
        for name in b:
            assert torch.equal(a[name], b[name]), name

    start, ws = i32([0, 9, 20]), B.topk_workspace(20, 30011, 40, "cuda", torch.bfloat16)
    outs = [{n: torch.zeros_like(v) for n, v in o.items()} for o in want]
    for o in (outs[0], outs[2]):
        o["grad"] = torch.zeros_like(x._base)[:, :30011]
    z = torch.zeros_like(x._base)
    zz = z[:, :30011]

    def step():
        B.dg_row_topk(zz, 40, ws=ws, out=outs[1])
        B.dg_distill_loss(zz, ii, tt, out=outs[0])
        B.dg_preference_loss(zz, tok, None, start, out=outs[2])
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    z.copy_(x._base)
    g.replay()
    for a, b in zip(outs, want):
        for name in b:
            assert torch.equal(a[name], b[name]), name


def test_calls_on_two_streams_do_not_disturb_each_other(B):
    """Kernels whose CTAs wait for one another, on streams that overlap, with a workspace each."""
    torch.manual_seed(3)
    V, K = 100003, 40
    x = torch.randn(300, 100004, device="cuda")[:, :V]
    top = B.dg_row_topk(x, K, lse=True)
    tok = torch.randint(0, V, (300,), device="cuda", dtype=torch.int32)
    adv = torch.randn(300, device="cuda")
    old = B.dg_token_logp(x, tok)["logp"] - 0.1

    def all_calls(ws, wk):
        d = B.dg_distill_loss(x, top["indices"], top["values"], top["lse"], temperature=1.5, grad=True, ws=ws)
        p = B.dg_policy_loss(x, tok, old, adv, grad=True, ws=ws)
        f = B.dg_token_logp(x, tok, temperature=0.8, ws=ws)
        t = B.dg_row_topk(x, K, lse=True, ws=wk)
        return [*d.values(), *p.values(), *f.values(), *t.values()]

    spaces = [(B.loss_workspace(300, V, x.device), B.topk_workspace(300, V, K, x.device)) for _ in range(2)]
    want = all_calls(*spaces[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    torch.cuda.synchronize()
    for rep in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(all_calls(*spaces[i]))
    torch.cuda.synchronize()
    B.dg_get_device_status()
    for runs in got:
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_directional_differences(B):
    """The forward call's losses along a direction against the gradient call: (f(x + hu) - f(x - hu)) / 2h
    with h = 2^-6: truncation h^2 / 6 of third derivatives below 1 per unit of sum |u|^3 p, rounding
    2 TOL / 2h; both below 2e-3 of a unit-scale derivative."""
    rng, x, xf, idx, t, lse = distill_case(8, 200, 12, "f32", 1.0, True)
    u = f32(rng.normal(0, 1, (8, 200)))
    h = 2.0 ** -6
    tok, one = i32(rng.integers(0, 200, 8)), f32(np.ones(8))
    logp = B.dg_token_logp(x, tok)["logp"]
    calls = {"distill": lambda y, **k: B.dg_distill_loss(y, i32(idx), f32(t), f32(lse), **k),
             "renormalised": lambda y, **k: B.dg_distill_loss(y, i32(idx), f32(t), **k),
             "policy": lambda y, **k: B.dg_policy_loss(y, tok, logp + 0.05, one, ref_logp=logp - 0.3, kl_coef=0.5, **k)}
    for name, f in calls.items():
        g = (f(x, grad=True)["grad"] * u).sum(1)
        d = (f(x + h * u)["loss"] - f(x - h * u)["loss"]) / (2 * h)
        near(d, g.double().cpu().numpy(), 2e-3 * (1 + g.abs().double().cpu().numpy()), name)


# --------------------------------------------------------------------------- top logits

TOPK = [(1, 1, 1), (3, 2, 2), (4, 37, 37), (2, 1000, 1), (5, 4097, 64), (3, 8192, 1024), (300, 257, 7), (2, 262144, 32),
        (1, 262144, 1000), (1, 1000, 1000), (33, 50001, 200), (160, 20000, 33), (2, 1000003, 100), (1, 2048, 1024),
        (700, 1100, 1024)]


@pytest.mark.parametrize("R,V,K", TOPK)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_topk(B, R, V, K, dtype):
    rng = np.random.default_rng(R + V + K)
    x, xf = logits(rng, R, V, dtype, 1, fill=float("inf"))
    check_topk(B, x, xf, K, 1.3)


def check_topk(B, x, xf, K, T=1.0):
    o = B.dg_row_topk(x, K, temperature=T, lse=True)
    want = L.row_topk(xf, K, T)
    assert np.array_equal(o["indices"].cpu().numpy(), want["indices"])
    assert np.array_equal(o["values"].double().cpu().numpy(), want["values"])
    near(o["lse"], want["lse"], tol_lse(xf, T), "lse")
    bare = B.dg_row_topk(x, K)
    assert torch.equal(bare["indices"], o["indices"]) and "lse" not in bare


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,K", [(300, 64), (33000, 64), (262144, 700)])
@pytest.mark.parametrize("shape", ["constant", "up", "down", "few values", "mostly -inf", "signed zeros", "steps", "lowest"])
def test_topk_orders(B, dtype, V, K, shape):
    """Ties, sorted rows (every entry a new maximum), rows with fewer finite entries than K."""
    rng = np.random.default_rng(V)
    i = np.arange(V)
    row = {"constant": lambda: np.full(V, 1.5),
           "up": lambda: i / V * 8 - 4,
           "down": lambda: 4 - i / V * 8,
           "few values": lambda: rng.integers(0, 4, V).astype(float),
           "mostly -inf": lambda: np.where(rng.random(V) < 20 / V, rng.normal(0, 1, V), -np.inf),
           "signed zeros": lambda: np.where(rng.random(V) < 0.5, 0.0, -0.0),
           "steps": lambda: (i // 2048) * 1.0,
           "lowest": lambda: np.where(i % 3 == 0, -3.3e38, -np.inf)}[shape]()
    if shape == "mostly -inf":
        row[V - 1] = 0.0      # at least one entry has mass
    x, xf = place(np.stack([row, row[::-1], np.roll(row, V // 3)]), dtype)
    o = B.dg_row_topk(x, K)
    want = L.row_topk(xf, K)
    assert np.array_equal(o["indices"].cpu().numpy(), want["indices"])
    assert np.array_equal(o["values"].double().cpu().numpy(), want["values"])


@pytest.mark.parametrize("R,V,K", [(700, 20000, 64), (310, 100003, 600), (1500, 3001, 300), (2048, 4096, 8), (400, 65536, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_topk_of_many_rows(B, R, V, K, dtype):
    """Several rows per CTA and rows that two CTAs share, in ascending order (the buffers of candidates fill
    up again and again) and at random, against a stable sort."""
    g = torch.Generator(device="cuda").manual_seed(R)
    x = torch.randn(R, (V + 7) // 8 * 8, device="cuda", generator=g)[:, :V]
    x[::3, :] = torch.arange(V, device="cuda") / V * 8 - 4
    x[1::6, V // 2:] = -float("inf")
    x = x.to(dtype)
    x = torch.nn.functional.pad(x, (0, -V % 8))[:, :V]
    o = B.dg_row_topk(x, K, lse=True)
    values, order = x.float().sort(dim=1, descending=True, stable=True)
    assert torch.equal(o["indices"].long(), order[:, :K]) and torch.equal(o["values"], values[:, :K])
    want = x.double().logsumexp(1)
    near(o["lse"], want.cpu().numpy(), tol_lse(x.double().cpu().numpy(), 1.0), "lse")


def test_topk_feeds_the_distillation(B):
    """The teacher's calls and the student's in a row: a teacher equal to the student has no loss."""
    rng = np.random.default_rng(11)
    x, xf = logits(rng, 64, 50001, "f32")
    top = B.dg_row_topk(x, 100, temperature=1.5, lse=True)
    o = B.dg_distill_loss(x, top["indices"], top["values"], top["lse"], temperature=1.5, grad=True)
    # q = p and q_0 = p_0 within 2 TOL + 100 u: the loss is of first order in that times nothing, of
    # second order otherwise; its terms round by 60 u each
    tl = 2 * tol_lse(xf, 1.5) + 200 * U
    near(o["loss"], np.zeros(64), 2.25 * 4 * tl, "loss")
    p = softmax(xf, 1.5)
    near(o["grad"], np.zeros_like(p), 1.5 * 4 * tl * p + 1e-30 + 1.5 * p * tl / np.exp(o["tail_logp"].double().cpu().numpy())[:, None],
         "gradient")


def test_indices_past_the_vocabulary_are_reported(B):
    from denoising_sampler_step_gb300.binding import DgError
    x, _ = logits(np.random.default_rng(0), 3, 100, "f32")
    for call in (lambda: B.dg_token_logp(x, i32([0, 100, 2])),
                 lambda: B.dg_token_logp_backward(x, i32([0, 1, 1 << 30]), f32([5, 5, 5]), f32([1, 1, 1])),
                 lambda: B.dg_distill_loss(x, i32([[0, 1], [2, 100], [3, 4]]), f32(np.zeros((3, 2))), grad=True)):
        call()
        with pytest.raises(DgError, match="past the vocabulary"):
            B.dg_get_device_status()
        B.dg_get_device_status()


def test_the_binding_refuses_wrong_tensors(B):
    x, _ = logits(np.random.default_rng(0), 3, 100, "f32")
    tok, one = i32([1, 2, 3]), f32([1, 1, 1])
    with pytest.raises(TypeError):
        B.dg_token_logp(x.half(), tok)
    with pytest.raises(ValueError):
        B.dg_token_logp(x.cpu(), tok)
    with pytest.raises(ValueError):
        B.dg_token_logp(x.t(), tok)
    with pytest.raises(ValueError):
        B.dg_token_logp(x, tok.long())
    with pytest.raises(ValueError):
        B.dg_token_logp(x, tok[:2])
    with pytest.raises(ValueError):
        B.dg_token_logp(x, tok, weight=one.cpu())
    with pytest.raises(ValueError):
        B.dg_token_logp(x, tok, weight=f32(np.ones(6))[::2])
    with pytest.raises(ValueError):
        B.dg_token_logp_backward(x, tok, one, one, out=x.bfloat16())
    with pytest.raises(ValueError):
        B.dg_distill_loss(x, i32([[1], [2]]), f32([[1], [2]]))
    with pytest.raises(ValueError):
        B.dg_preference_loss(x, tok, one, i32([0, 1]))
    with pytest.raises(B.DgError):
        B.dg_token_logp(x[:, 1:], tok)      # rows off a 16-byte boundary
    with pytest.raises(B.DgError):
        B.dg_row_topk(x, 101)
