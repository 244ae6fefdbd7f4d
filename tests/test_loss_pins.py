"""The loss oracle against closed forms and central differences, and the loss calls' refusals on
the host (no GPU)."""
import ctypes

import numpy as np
import pytest

from oracle import loss_oracle as L

H = 1e-5
# central differences in float64: truncation H^2 |f'''| / 6 ~ 1e-11, rounding 1e-16 |f| / H ~ 1e-11;
# two digits of room
DIFF_TOL = 1e-8


def differences(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += H
        down[i] -= H
        g[i] = (f(up) - f(down)) / (2 * H)
    return g


@pytest.fixture
def rows():
    rng = np.random.default_rng(7)
    return rng, rng.normal(0, 2, (5, 11)), np.array([0.3, 1.0, 0.0, 0.7, 2.0])


@pytest.mark.parametrize("T", [1.0, 1.7])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_by_differences(rows, T, tail):
    rng, x, w = rows
    t_all = rng.normal(0, 2, x.shape)
    top = L.row_topk(t_all, 4, T)
    idx = top["indices"].copy()
    idx[1, 2] = -1
    lse = top["lse"] if tail else None
    args = (idx, top["values"], lse, T, w)
    g = L.distill_loss(x, *args)["grad"]
    d = differences(lambda y: float(w @ L.distill_loss(y, *args)["loss"]), x)
    assert np.abs(g - d).max() < DIFF_TOL
    assert not g[2].any()


@pytest.mark.parametrize("T", [1.0, 0.6])
@pytest.mark.parametrize("kl_coef", [0.0, 0.3])
def test_policy_gradient_by_differences(rows, T, kl_coef):
    rng, x, w = rows
    tok = np.array([0, 10, 3, -1, 5])
    logp = L.token_logp(x, np.maximum(tok, 0), T)["logp"]
    # ratios on every side of the clipping range, away from its ends
    old = logp - np.log([0.5, 1.5, 1.0, 1.0, 1.05])
    A = np.array([1.0, 2.0, 1.0, 1.0, -0.7])
    kw = dict(ref_logp=logp + 0.3, clip_low=0.2, clip_high=0.3, kl_coef=kl_coef, T=T, weight=w)
    g = L.policy_loss(x, tok, old, A, **kw)["grad"]
    d = differences(lambda y: float(w @ L.policy_loss(y, tok, old, A, **kw)["loss"]), x)
    assert np.abs(g - d).max() < DIFF_TOL
    assert list(L.policy_loss(x, tok, old, A, **kw)["clipped"]) == [0, 1, 0, 0, 0]


@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_preference_gradient_by_differences(rows, smoothing):
    rng, x, w = rows
    tok = np.array([0, 10, 3, -1, 5])
    start, pw = np.array([0, 2, 2, 3, 5]), np.array([0.5, 2.0])
    ref = rng.normal(-3, 1, 5)
    kw = dict(beta=0.4, label_smoothing=smoothing, T=1.3, weight=w, pair_weight=pw)
    g = L.preference_loss(x, tok, ref, start, **kw)["grad"]
    d = differences(lambda y: float(pw @ L.preference_loss(y, tok, ref, start, **kw)["loss"]), x)
    assert np.abs(g - d).max() < DIFF_TOL


def test_closed_forms():
    x = np.log(np.array([[1.0, 2.0, 5.0]]))
    assert np.allclose(L.token_logp(x, [1])["logp"], np.log(0.25))
    # a teacher equal to the student: no divergence, no gradient, with and without the bucket
    top = L.row_topk(x, 3)
    for lse in (None, top["lse"]):
        o = L.distill_loss(x, top["indices"], top["values"], lse)
        assert abs(o["loss"][0]) < 1e-15 and np.abs(o["grad"]).max() < 1e-15
    top = L.row_topk(x, 2)
    o = L.distill_loss(x, top["indices"], top["values"], top["lse"])
    assert abs(o["loss"][0]) < 1e-15 and np.abs(o["grad"]).max() < 1e-15
    assert np.allclose(o["tail_logp"], np.log(1 / 8))
    # over the two renormalised entries: -ln of their share, 7/8
    assert np.allclose(L.distill_loss(x, top["indices"], top["values"])["loss"], -np.log(7 / 8))
    # ratio 1: the loss is -A, the derivative -A
    o = L.policy_loss(x, [2], [np.log(5 / 8)], [3.0], ref_logp=[np.log(5 / 8)], kl_coef=1.0)
    assert np.allclose(o["loss"], -3) and np.allclose(o["dlogp"], -3) and o["clipped"][0] == 0
    # equal sequences: ln 2
    o = L.preference_loss(np.repeat(x, 2, 0), [1, 1], None, [0, 1, 2])
    assert np.allclose(o["loss"], np.log(2)) and np.allclose(o["dlogp"], [-0.05, 0.05])
    assert np.allclose(L.preference_loss(x[:0], np.zeros(0, int), None, [0, 0, 0])["loss"], np.log(2))


def test_topk_order_of_ties():
    x = np.array([[0.0, -0.0, 1.0, -np.inf, 1.0]])
    assert list(L.row_topk(x, 5)["indices"][0]) == [2, 4, 0, 1, 3]


# --------------------------------------------------------------------------- refusals on the host

@pytest.fixture(scope="module")
def lib():
    from denoising_sampler_step_gb300 import build
    build.build()
    from denoising_sampler_step_gb300 import binding
    return binding.lib


P, Q, BIG = ctypes.c_void_p(256), ctypes.c_void_p(264), ctypes.c_void_p(1 << 40)
ROWS = [P, 0, 4, 100, 100]


WS = [P, 1 << 30, None]    # workspace, its size, stream


NAMES = ("topk", "logp", "logp_bwd", "distill", "distill_bwd", "policy", "pref")


def calls(lib, rows, T=1.0, grad=BIG, ldg=100, K=5, ldk=5, ws=WS, names=NAMES):
    """The named calls of this part on the same rows: status by name.  Only calls that must be refused are
    made: the pointers are made up."""
    f = {
        "topk": lambda: lib.dg_row_topk(*rows, K, T, P, P, ldk, P, *ws),
        "logp": lambda: lib.dg_token_logp(*rows, P, T, None, P, P, *ws),
        "logp_bwd": lambda: lib.dg_token_logp_backward(*rows, P, T, P, P, None, grad, ldg, *ws),
        "distill": lambda: lib.dg_distill_loss(*rows, P, P, K, ldk, None, T, None, P, P, P, grad, ldg, *ws),
        "distill_bwd": lambda: lib.dg_distill_loss_backward(*rows, P, P, K, ldk, None, T, P, None, None, grad, ldg, *ws),
        "policy": lambda: lib.dg_policy_loss(*rows, P, P, P, P, T, 0.2, 0.2, 0.0, None, *([P] * 6), grad, ldg, *ws),
        "pref": lambda: lib.dg_preference_loss(*rows, P, P, P, 1, 0.1, 0.0, T, None, None, *([P] * 5), grad, ldg, *ws),
    }
    return {n: f[n]() for n in names}


@pytest.mark.parametrize("rows,status", [
    ([P, 2, 4, 100, 100], 1),              # unknown dtype
    ([P, 0, -1, 100, 100], 1),
    ([P, 0, 4, 0, 100], 1),
    ([P, 0, 4, 100, 96], 1),               # ldl < V
    ([None, 0, 4, 100, 100], 1),
    ([Q, 0, 4, 100, 100], 2),              # base not 16-byte aligned
    ([P, 0, 4, 100, 101], 2),              # rows not 16-byte aligned
    ([P, 1, 4, 100, 100], 2),              # bf16 needs ldl % 8 == 0
    ([P, 0, 4, 0x7ffffff4, 0x7ffffff4], 2),
    ([P, 0, 1 << 28, 100, 1 << 40], 2),    # offsets past 64 bits
    ([P, 0, 1 << 29, 100, 100], 2),
])
def test_calls_refuse_bad_rows(lib, rows, status):
    for name, st in calls(lib, rows).items():
        assert st == status, name


@pytest.mark.parametrize("T", [0.0, -1.0, float("inf"), float("nan")])
def test_calls_refuse_bad_temperatures(lib, T):
    for name, st in calls(lib, ROWS, T=T).items():
        assert st == 1, name
        assert b"temperature" in lib.dg_last_error()


@pytest.mark.parametrize("grad,ldg,status", [
    (BIG, 96, 1), (BIG, 102, 2), (ctypes.c_void_p((1 << 40) + 8), 100, 2),
    (P, 104, 1),                           # on the logits with another stride
    (ctypes.c_void_p(256 + 16), 100, 1),   # overlapping them
    (ctypes.c_void_p(256 + 1584), 100, 1), (BIG, 1 << 55, 2)])
def test_calls_refuse_bad_gradients(lib, grad, ldg, status):
    for name, st in calls(lib, ROWS, grad=grad, ldg=ldg, names=NAMES[2:]).items():
        assert st == status, name


def test_backward_calls_need_a_gradient_and_saved_values(lib):
    rows = ROWS
    assert lib.dg_token_logp_backward(*rows, P, 1.0, P, P, None, None, 100, *WS) == 1
    assert lib.dg_token_logp_backward(*rows, P, 1.0, None, P, None, BIG, 100, *WS) == 1
    assert lib.dg_token_logp_backward(*rows, P, 1.0, P, None, None, BIG, 100, *WS) == 1
    assert lib.dg_distill_loss_backward(*rows, P, P, 5, 5, None, 1.0, P, None, None, None, 100, *WS) == 1
    assert lib.dg_distill_loss_backward(*rows, P, P, 5, 5, None, 1.0, None, None, None, BIG, 100, *WS) == 1
    assert lib.dg_distill_loss_backward(*rows, P, P, 5, 5, P, 1.0, P, None, None, BIG, 100, *WS) == 1
    assert b"tail_logp" in lib.dg_last_error()


@pytest.mark.parametrize("K,ldk,status", [(0, 5, 1), (5, 4, 1), (1025, 1025, 2), (5, 1 << 33, 2)])
def test_calls_refuse_bad_entry_tables(lib, K, ldk, status):
    rows = [P, 0, 4, 2000, 2000]
    for name, st in calls(lib, rows, ldg=2000, K=K, ldk=ldk, names=("topk", "distill", "distill_bwd")).items():
        assert st == status, name


def test_topk_refuses_more_entries_than_columns_and_a_small_workspace(lib):
    assert lib.dg_row_topk(*ROWS, 101, 1.0, P, P, 101, P, P, 1 << 30, None) == 1
    assert lib.dg_row_topk(*ROWS, 5, 1.0, None, P, 5, P, P, 1 << 30, None) == 1
    assert lib.dg_row_topk_workspace_size(4, 100, 101, 0) == 0
    assert lib.dg_row_topk_workspace_size(4, 100, 5, 7) == 0
    assert lib.dg_row_topk_workspace_size(0, 100, 5, 0) == 0


def test_losses_refuse_a_small_or_unaligned_workspace(lib):
    assert lib.dg_row_loss_workspace_size(4, 100, 2) == 0 and lib.dg_row_loss_workspace_size(0, 9, 0) == 0
    bad = lambda need: ((None, 1 << 30, 1), (P, need - 1, 1), (Q, 1 << 30, 2))
    need = lib.dg_row_loss_workspace_size(4, 20000, 0)
    assert need > 0 and lib.dg_row_loss_needs_workspace(20000, 0) == 1
    for ws, n, status in bad(need):
        for name, st in calls(lib, [P, 0, 4, 20000, 20000], ldg=20000, ws=[ws, n, None], names=NAMES[1:]).items():
            assert st == status, (name, st)
    # rows of one tile take a workspace in one call only
    need = lib.dg_row_loss_workspace_size(4, 100, 0)
    assert need > 0 and lib.dg_row_loss_needs_workspace(100, 0) == 0
    for ws, n, status in bad(need):
        assert lib.dg_distill_loss_backward(*ROWS, P, P, 5, 5, None, 1.0, P, None, None, BIG, 100, ws, n, None) == status
    assert [lib.dg_row_loss_needs_workspace(16384 + 4 * i, 0) for i in (0, 1)] == [0, 1]
    assert [lib.dg_row_loss_needs_workspace(32768 + 8 * i, 1) for i in (0, 1)] == [0, 1]
    assert lib.dg_row_loss_needs_workspace(1 << 20, 2) == 0


def test_policy_refuses_bad_coefficients(lib):
    def call(lo=0.2, hi=0.2, kl=0.0, tok=P, old=P, adv=P):
        return lib.dg_policy_loss(*ROWS, tok, old, None, adv, 1.0, lo, hi, kl, None, *([P] * 6), None, 0, *WS)
    nan, inf = float("nan"), float("inf")
    for bad in (dict(lo=-0.1), dict(lo=1.1), dict(lo=nan), dict(hi=-0.1), dict(hi=inf), dict(hi=nan), dict(kl=-1.0),
                dict(kl=inf), dict(kl=nan), dict(tok=None), dict(old=None), dict(adv=None)):
        assert call(**bad) == 1, bad


def test_preference_refuses_bad_pairs(lib):
    def call(pairs=1, beta=0.1, eps=0.0, start=P, loss=P, dlogp=P):
        return lib.dg_preference_loss(*ROWS, P, P, start, pairs, beta, eps, 1.0, None, None, loss, P, P, P, dlogp,
                                      None, 0, *WS)
    nan, inf = float("nan"), float("inf")
    for bad in (dict(pairs=-1), dict(beta=inf), dict(beta=nan), dict(eps=-0.1), dict(eps=1.0), dict(eps=nan),
                dict(start=None), dict(loss=None), dict(dlogp=None)):
        assert call(**bad) == 1, bad


def test_no_rows_queue_nothing(lib):
    rows = [None, 0, 0, 100, 100]
    assert lib.dg_row_topk(*rows, 5, 1.0, None, None, 5, None, None, 0, None) == 0
    assert lib.dg_token_logp(*rows, None, 1.0, None, None, None, None, 0, None) == 0
    assert lib.dg_token_logp_backward(*rows, None, 1.0, None, None, None, None, 100, None, 0, None) == 0
    assert lib.dg_distill_loss(*rows, None, None, 5, 5, None, 1.0, None, None, None, None, None, 100, None, 0, None) == 0
    assert lib.dg_distill_loss_backward(*rows, None, None, 5, 5, None, 1.0, None, None, None, None, 100, None, 0, None) == 0
    assert lib.dg_policy_loss(*rows, None, None, None, None, 1.0, 0.2, 0.2, 0.0, None, *([None] * 7), 100, None, 0, None) == 0
    assert lib.dg_preference_loss(*rows, None, None, None, 0, 0.1, 0.0, 1.0, None, None, *([None] * 6), 100,
                                  None, 0, None) == 0
