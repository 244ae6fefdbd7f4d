"""The hidden stream's calls at batch sizes, against float64 on the GPU: norms with two, four and eight eights of columns a
thread over several turns of every CTA, gradients of wide tables and of more than 65,536 positions, the head's resident
positions over many tiles, and matrices of more than 2^31 entries.  Tolerances as in test_gpu_hidden.py."""
import numpy as np
import pytest
import torch

from test_gpu_hidden import B, HALF, T, U, check_head, device_status_stays_clear  # noqa: F401

pytestmark = pytest.mark.gpu


def rows(g, R, d, kind, size=None):
    """Random rows on 16-byte boundaries."""
    per = 16 // T[kind].itemsize
    out = torch.empty(R, (d + per - 1) // per * per, dtype=T[kind], device="cuda")[:, :d]
    step = max(1, (1 << 27) // d)
    for i in range(0, R, step):
        x = torch.randn(min(step, R - i), d, generator=g, device="cuda")
        out[i:i + step] = x if size is None else x * size[i:i + step]
    return out


def check_norm(x, residual, w, o, at, eps=1e-6):
    """Rows `at` of dg_rms_norm's 8-bit output with hidden kept."""
    h = x[at].double() + residual[at].double()
    rstd = (h.square().mean(1) + eps) ** -0.5
    y = h * rstd[:, None] * w
    assert ((o["hidden"][at] - h).abs() <= U * h.abs()).all()
    assert ((o["rstd"][at] - rstd).abs() <= 52 * U * rstd).all()
    s, top = o["scale"][at].double()[:, None], y.abs().amax(1, keepdim=True)
    assert ((s - top / 448).abs() <= 57 * U * top / 448).all()
    q = o["out"][at].view(torch.float8_e4m3fn).double() * s
    assert ((q - y).abs() <= torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s) * (1 + 4 * U) + 60 * U * y.abs()).all()


def check_gradient(grad, hidden, rstd, w, up, got, at, kind):
    """Rows `at` of dg_rms_norm_backward's gradient; what they add to the weight's, and the magnitudes of that."""
    xh, g = hidden[at].double() * rstd[at].double()[:, None], grad[at].double()
    rs, gw = rstd[at].double()[:, None], g * w
    inner, size = (gw * xh).mean(1, keepdim=True), (gw * xh).abs().mean(1, keepdim=True)
    ref = rs * (gw - xh * inner)
    tol = rs * (6 * U * gw.abs() + 102 * U * xh.abs() * size)
    if up is not None:
        ref = ref + up[at].double()
        tol = tol + U * up[at].double().abs()
    assert ((got[at].double() - ref).abs() <= tol + (HALF[kind] + 2 * U) * ref.abs()).all()
    return (g * xh).sum(0), (g * xh).abs().sum(0)


@pytest.mark.parametrize("R,d", [(5003, 1153), (8192, 2816), (3001, 4104), (2500, 8200), (500, 20001)])
@pytest.mark.parametrize("x,up", [("bf16", "bf16"), ("f32", None), ("bf16", "f32")])
def test_norm_and_its_gradient_over_many_rows(B, R, d, x, up):
    g = torch.Generator(device="cuda").manual_seed(R)
    size = torch.exp(torch.randn(R, 1, generator=g, device="cuda"))
    xt, rt = rows(g, R, d, x, size), rows(g, R, d, "f32", size)
    w = (0.3 * torch.randn(d, generator=g, device="cuda")).to(T[x])
    wd = 1.0 + w.double()
    o = B.dg_rms_norm(xt, w, residual=rt, weight_offset=1.0, dtype=torch.uint8)
    at = [slice(i, i + 500) for i in range(0, R, 500)]
    for i in at:
        check_norm(xt, rt, wd, o, i)
    y = B.dg_rms_norm(xt, w, residual=rt, weight_offset=1.0, dtype=T[x])
    assert torch.equal(y["rstd"], o["rstd"]) and torch.equal(y["hidden"], o["hidden"])
    for i in at:
        h = xt[i].double() + rt[i].double()
        want = h * ((h.square().mean(1, keepdim=True) + 1e-6) ** -0.5) * wd
        assert ((y["out"][i].double() - want).abs() <= (56 * U + HALF[x]) * want.abs()).all()
    grad, ut = rows(g, R, d, x), rows(g, R, d, up) if up else None
    hid = xt if x == "bf16" else o["hidden"]
    rstd = (hid.double().square().mean(1) + 1e-6).rsqrt().float()
    b = B.dg_rms_norm_backward(grad, hid, rstd, w, 1.0, grad_hidden=ut)
    sums = [check_gradient(grad, hid, rstd, wd, ut, b["grad"], i, x) for i in at]
    want, terms = (sum(s[k] for s in sums) for k in (0, 1))
    assert ((b["grad_weight"].double() - want).abs() <= (R + 3) * U * terms + HALF[x] * want.abs()).all()


@pytest.mark.parametrize("R,V,d", [(300, 900, 1025), (700, 300, 1025), (6001, 9000, 2816), (3000, 500, 8200), (30000, 4000, 1100),
                                   (66001, 20000, 300), (70001, 40000, 1030)])
@pytest.mark.parametrize("gt,tt", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("kind", ["text", "masked"])
def test_gradient_of_wide_tables(B, R, V, d, gt, tt, kind):
    g = torch.Generator(device="cuda").manual_seed(R + d)
    grad = rows(g, R, d, gt)
    if kind == "text":
        tok = torch.exp(torch.rand(R, generator=g, device="cuda") * np.log(V + 1.0)).long().clamp(1, V) - 1
    else:
        tok = torch.randint(V, (R,), generator=g, device="cuda")
        tok[torch.rand(R, generator=g, device="cuda") < 0.6] = V // 3
    tok[torch.rand(R, generator=g, device="cuda") < 0.1] = -1
    on = tok >= 0
    at = tok.clamp(min=0)
    n = torch.zeros(V, device="cuda", dtype=torch.float64).index_add_(0, at, on.double())[:, None]
    add = lambda x: torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, at, x * on[:, None])  # noqa: E731
    want, size = 16.0 * add(grad.double()), 16.0 * add(grad.double().abs())
    tok = tok.int()
    got = B.dg_token_embed_backward(grad, tok, V, 16.0, dtype=T[tt])
    assert ((got.double() - want).abs() <= (n + 3) * U * size + HALF[tt] * want.abs()).all()
    assert torch.equal(got, B.dg_token_embed_backward(grad, tok, V, 16.0, dtype=T[tt]))
    old = rows(g, V, d, tt)
    total = want + old.double()
    new = B.dg_token_embed_backward(grad, tok, V, 16.0, accumulate=True, out=old.clone())
    tol = (n + 3) * U * size + U * old.double().abs() + (U + HALF[tt]) * total.abs()
    assert ((new.double() - total).abs() <= tol).all()
    assert torch.equal(new[n[:, 0] == 0], old[n[:, 0] == 0])


@pytest.mark.parametrize("R,V,d", [(200, 60001, 80), (100, 50004, 300), (65, 80000, 16), (256, 40008, 600), (256, 41000, 800)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_head_with_few_positions_over_many_tiles(B, R, V, d, out):
    check_head(B, R, V, d, out)


# --------------------------------------------------------------------------- more than 2^31 entries

def test_norms_past_32_bits(B):
    R, d = 770_000, 2816                                       # 2.17e9 entries
    g = torch.Generator(device="cuda").manual_seed(4)
    x, res = rows(g, R, d, "bf16"), rows(g, R, d, "f32")
    w = torch.randn(d, generator=g, device="cuda")
    o = B.dg_rms_norm(x, w, residual=res, dtype=torch.uint8)
    past = (1 << 31) // d                                      # the row in which entry 2^31 lies
    for i in (slice(0, 300), slice(R // 2, R // 2 + 300), slice(past - 150, past + 150), slice(R - 300, R)):
        check_norm(x, res, w.double(), o, i)
    del res
    # the gradient of all rows: its weight's is a sum over them
    b = B.dg_rms_norm_backward(x, o["hidden"], o["rstd"], w, grad_hidden=x)
    want, terms = torch.zeros(2, d, dtype=torch.float64, device="cuda")
    for i in range(0, R, 20000):
        s, t = check_gradient(x, o["hidden"], o["rstd"], w.double(), x, b["grad"], slice(i, i + 20000), "f32")
        want += s
        terms += t
    assert ((b["grad_weight"] - want).abs() <= (R + 3) * U * terms + U * want.abs()).all()


def test_gradient_of_rows_past_32_bits(B):
    R, V, d = 770_000, 1000, 2816
    g = torch.Generator(device="cuda").manual_seed(5)
    grad = rows(g, R, d, "bf16")
    tok = torch.randint(V, (R,), generator=g, device="cuda").int()
    got = B.dg_token_embed_backward(grad, tok, V, 1.0, dtype=torch.float32)
    want, size = torch.zeros(2, V, d, dtype=torch.float64, device="cuda")
    for i in range(0, R, 50000):
        want.index_add_(0, tok[i:i + 50000], grad[i:i + 50000].double())
        size.index_add_(0, tok[i:i + 50000], grad[i:i + 50000].double().abs())
    n = torch.bincount(tok, minlength=V)[:, None]
    assert ((got - want).abs() <= (n + 3) * U * size).all()


@pytest.mark.parametrize("R,V,out", [(8200, 262152, "bf16"), (130, 16_600_000, "f32")])
def test_logits_past_32_bits(B, R, V, out):
    d = 48
    g = torch.Generator(device="cuda").manual_seed(6)

    def codes(n):
        x = 4.0 * torch.randn(n, d, generator=g, device="cuda")
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    X, Q = codes(R), codes(V)
    xs, s = 0.5 + torch.rand(R, generator=g, device="cuda"), 1e-3 * (1 + torch.rand(V, generator=g, device="cuda"))
    o = B.dg_head_e4m3(X, xs, Q, s, dtype=T[out])
    x, q = (t.view(torch.float8_e4m3fn).double() * f.double()[:, None] for t, f in ((X, xs), (Q, s)))
    step = max(1, (1 << 27) // V)
    for i in sorted({0, R // 2, (1 << 31) // V, R - step, *range(0, R, max(step, R // 6))}):
        a = x[i:i + step]
        ref, terms = a @ q.T, a.abs() @ q.abs().T
        tol = (d / 32 + 33) * 2.0 ** -23 * terms + (3 * U + HALF[out]) * ref.abs()
        assert ((o[i:i + step].double() - ref).abs() <= tol).all(), i
