"""The hidden stream's calls against the float64 oracle (oracle/hidden_oracle.py).

Tolerances, derived from fp32 (u = 2^-24) before the kernels ran; `half` is half a step of the output's type,
u (fp32), 2^-9 of the value's power of two, so at most 2^-8 of the value, (bf16):

* lookup: an entry times its scale times gamma, three roundings: 3 u of the value, and half.
* the table's gradient: n terms of a token added in some order, gamma and what was there: (n + 3) u times the
  terms' magnitudes, u of the old value, and half.
* a norm: a sum of squares of d terms in at most 96 levels (8 per group, up to 4 groups, 5 shuffles, up to 32
  warps, and one for each of mean, eps, root, quotient), halved by the root: rstd within 52 u, and y = h rstd w
  with four more: 56 u of y, and half.  h is one rounding.
* 8 bits: scale = max / 448 within 57 u.  A code is the nearest to y / scale: half a step of E4M3 (2^-4 of the
  value, 2^-10 for subnormal codes, times scale), and y's own 56 u and the quotient's.
* the norm's gradient: inner sums as above, 96 u of the terms' magnitudes; each term of dh carries its factors'
  roundings, six u in all; dweight is R terms in some order, (R + 3) u of their magnitudes; and half.
* the head: products of codes are exact; every step of 32 terms rounds or cuts the running fp32 sum and its own
  terms at no more than 2^-23 of the largest of them: (d / 32 + 33) 2^-23 of the terms' magnitudes, three u, half.
"""
import numpy as np
import pytest
import torch

from oracle import e4m3_decode, hidden_oracle as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
T = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}
HALF = {"f32": U, "bf16": 2.0 ** -8}
FILL = {"f32": -777.0, "bf16": -776.0, "e4m3": 0x7F}   # what lies beside a matrix; not to be read or written


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


def place(x, kind, layout="wide"):
    """(tensor of x's values rounded to the type, those values in float64).  layouts: rows on 16-byte boundaries with
    columns beside them (wide), one after another (dense), off any 16-byte boundary (odd)."""
    x = torch.as_tensor(np.asarray(x))
    R, d = x.shape
    per = 16 // T[kind].itemsize
    lead, ld = {"wide": (0, (d + per - 1) // per * per + per), "dense": (0, d), "odd": (1, d + 3)}[layout]
    buf = torch.full((lead + R * ld + 64,), FILL[kind], dtype=T[kind], device="cuda")
    view = buf[lead:lead + R * ld].view(R, ld)[:, :d]
    view.copy_(x.to(T[kind]))
    view.around = buf
    return view, (view.cpu().numpy() if kind == "e4m3" else view.double().cpu().numpy())


def empty(R, d, kind, layout="wide"):
    return place(np.full((R, d), 3 if kind == "e4m3" else 3.0), kind, layout)[0]


def untouched(view, kind):
    """Nothing beside the matrix was written."""
    R, d = view.shape
    buf = view.around.clone()
    lead = view.storage_offset()
    buf[lead:lead + R * view.stride(0)].view(R, view.stride(0))[:, :d] = FILL[kind]
    assert (buf == FILL[kind]).all()


def close(got, ref, tol):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size}: off by {np.abs(got - ref)[bad].max()} against {np.broadcast_to(tol, ref.shape)[bad].min()}"


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def f32(a):
    return torch.as_tensor(np.asarray(a, np.float32)).cuda()


def tokens(rng, kind, R, V):
    t = rng.integers(0, V, R)
    if kind == "one":
        t[:] = V // 2
    elif kind == "masked":
        t[rng.random(R) < 0.6] = V - 1
    elif kind == "distinct":
        t = rng.permutation(np.arange(max(R, V)))[:R] % V
    elif kind == "runs":  # lengths around every size of a unit, in shuffled places
        n = rng.integers(1, 140, R)
        t = rng.permutation(np.repeat(rng.permutation(np.arange(R)) % V, n)[:R])
    elif kind == "padded":
        t[rng.random(R) < 0.4] = -1
        t[: R // 8] = -2 ** 31
    return t.astype(np.int32)


# --------------------------------------------------------------------------- lookup

SHAPES = [(1, 10, 1), (5, 7, 3), (16, 4096, 256), (33, 1000, 255), (7, 50, 2817), (300, 500, 1001), (1025, 100, 8),
          (2, 3, 8200)]


@pytest.mark.parametrize("R,V,d", SHAPES)
@pytest.mark.parametrize("table,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("e4m3", "bf16"), ("e4m3", "f32")])
@pytest.mark.parametrize("layout", ["wide", "dense", "odd"])
def test_lookup(B, R, V, d, table, out, layout):
    rng = np.random.default_rng(R + d)
    scale = rng.uniform(1e-4, 3e-4, V).astype(np.float32)
    if table == "e4m3":
        Wd, codes = place(rng.choice(np.delete(np.arange(256), [0x7F, 0xFF]), (V, d)).astype(np.uint8), table, layout)
        W = e4m3_decode(codes) * scale[:, None].astype(np.float64)
    else:
        Wd, W = place(rng.normal(size=(V, d)), table, layout)
    tok = tokens(rng, "padded", R, V)
    o = empty(R, d, out, layout)
    got = B.dg_token_embed(Wd, i32(tok), 53.0, scale=f32(scale) if table == "e4m3" else None, out=o)
    assert got is o
    ref = H.token_embed(W, tok, 53.0)
    close(o, ref, (3 * U + HALF[out]) * np.abs(ref))
    untouched(o, out)


def test_slices_of_the_vocabulary(B):
    rng = np.random.default_rng(1)
    W, tok = rng.normal(size=(1000, 40)), tokens(rng, "padded", 500, 1000)
    whole = None
    for a, b in ((0, 250), (250, 250), (250, 611), (611, 1000)):
        Wd, Wv = place(np.concatenate([W[a:b], np.full((3, 40), np.nan)]), "bf16")    # padding rows are never read
        got = B.dg_token_embed(Wd, i32(tok), 2.0, vocab_start=a, vocab_end=b, V=1000, dtype=torch.float32)
        close(got, H.token_embed(Wv[:b - a], tok, 2.0, a, b), 0.0)   # a bf16 value times 2
        whole = got if whole is None else whole + got
    Wd, _ = place(W, "bf16")
    assert torch.equal(whole, B.dg_token_embed(Wd, i32(tok), 2.0, dtype=torch.float32))


def test_tokens_past_the_vocabulary(B):
    Wd, W = place(np.ones((8, 16)), "f32")
    tok = [0, 8, 7, 2 ** 31 - 1, -5]
    got = B.dg_token_embed(Wd, i32(tok), 1.0)
    with pytest.raises(B.DgError, match="INVALID_ARG"):
        B.dg_get_device_status()
    assert got.sum(1).tolist() == [16, 0, 16, 0, 0]
    g = B.dg_token_embed_backward(torch.ones(5, 16, device="cuda"), i32(tok), 8)
    with pytest.raises(B.DgError, match="INVALID_ARG"):
        B.dg_get_device_status()
    assert g.sum(1).tolist() == [16, 0, 0, 0, 0, 0, 0, 16]


def test_a_table_past_32_bits(B):
    V, d = 1 << 21, 1040                                   # 2.2e9 codes
    Q = torch.zeros(V, d, dtype=torch.uint8, device="cuda")
    Q[-3:] = 0x38                                          # 1
    tok = [V - 1, V - 3, V - 4, 0]
    got = B.dg_token_embed(Q, i32(tok), 3.0, scale=torch.full((V,), 0.5, device="cuda"))
    assert (got[:2] == 1.5).all() and not got[2:].any()
    del Q
    grad = torch.zeros(V, d, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(4, d, dtype=torch.bfloat16, device="cuda")
    B.dg_token_embed_backward(g, i32(tok), V, 2.0, accumulate=True, out=grad)
    assert grad.count_nonzero() == 4 * d and (grad[[V - 1, V - 3, V - 4, 0]] == 2).all()


# --------------------------------------------------------------------------- its gradient

@pytest.mark.parametrize("kind", ["uniform", "one", "masked", "distinct", "runs", "padded"])
@pytest.mark.parametrize("R,V,d", [(1, 5, 8), (9, 4, 1), (64, 70, 257), (300, 40, 33), (2047, 3000, 40), (2049, 300, 8),
                                   (8200, 20000, 16), (33000, 600, 9), (70001, 70000, 3)])
def test_gradient(B, R, V, d, kind):
    rng = np.random.default_rng(R)
    dt, tt = ("f32", "bf16") if R % 2 else ("bf16", "f32")
    tok = tokens(rng, kind, R, V)
    gd, g = place(rng.normal(size=(R, d)), dt, "odd" if d % 8 else "wide")
    o = empty(V, d, tt)
    ws = torch.full((B.dg_token_embed_backward_workspace_size(R, V, d) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    B.dg_token_embed_backward(gd, i32(tok), V, 16.0, out=o, ws=ws[:-64])
    assert (ws[-64:] == 0xFF).all()
    untouched(o, tt)
    ref = H.token_embed_backward(g, tok, 16.0, 0, V)
    tol = (ref["count"] + 3)[:, None] * U * ref["size"]
    close(o, ref["grad"], tol + HALF[tt] * np.abs(ref["grad"]))
    again = empty(V, d, tt)
    B.dg_token_embed_backward(gd, i32(tok), V, 16.0, out=again, ws=ws[:-64])
    assert torch.equal(again, o)                            # bit for bit
    # added to what is there; rows of tokens that do not occur stay as they were, NaN included
    old = rng.normal(size=(V, d))
    old[ref["count"] == 0] = np.nan
    ad, a = place(old, tt)
    before = ad.clone()
    B.dg_token_embed_backward(gd, i32(tok), V, 16.0, accumulate=True, out=ad, ws=ws[:-64])
    untouched(ad, tt)
    there = ref["count"] > 0
    total = (a + ref["grad"])[there]
    close(ad[torch.as_tensor(there).cuda()], total, tol[there] + U * np.abs(a[there]) + (U + HALF[tt]) * np.abs(total))
    assert torch.equal(ad.view(torch.int16 if tt == "bf16" else torch.int32)[torch.as_tensor(~there).cuda()],
                       before.view(torch.int16 if tt == "bf16" else torch.int32)[torch.as_tensor(~there).cuda()])


# where the order of the tokens is found in another way, or in one run, or one position, more
@pytest.mark.parametrize("kind", ["uniform", "masked"])
@pytest.mark.parametrize("R,V,d", [(256, 70, 5), (257, 70, 5), (512, 70, 5), (513, 70, 5), (1025, 9, 8), (2048, 700, 8), (4097, 33, 8), (24575, 50, 8),
                                   (24576, 9000, 8), (24577, 50, 8), (65536, 1000, 8), (65537, 1000, 8)])
def test_gradient_where_the_order_changes(B, R, V, d, kind):
    test_gradient(B, R, V, d, kind)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("tt", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["wide", "dense", "odd"])
def test_gradients_types_and_strides(B, dt, tt, layout):
    rng = np.random.default_rng(3)
    tok = tokens(rng, "masked", 500, 90)
    gd, g = place(rng.normal(size=(500, 261)), dt, layout)
    o = empty(90, 261, tt, layout)
    B.dg_token_embed_backward(gd, i32(tok), 90, 0.37, out=o)
    untouched(o, tt)
    ref = H.token_embed_backward(g, tok, 0.37, 0, 90)
    # (gamma as the fp32 number that the call takes: another u)
    close(o, ref["grad"], (ref["count"] + 4)[:, None] * U * ref["size"] + HALF[tt] * np.abs(ref["grad"]))


def test_gradient_of_a_slice(B):
    rng = np.random.default_rng(4)
    tok = tokens(rng, "padded", 700, 1000)
    gd, g = place(rng.normal(size=(700, 24)), "f32")
    for a, b in ((0, 1000), (0, 1), (313, 900), (999, 1000), (500, 500)):
        o = empty(b - a + 2, 24, "f32")                     # two rows of padding: not written
        B.dg_token_embed_backward(gd, i32(tok), 1000, 1.0, vocab_start=a, vocab_end=b, out=o)
        ref = H.token_embed_backward(g, tok, 1.0, a, b)
        close(o[:b - a], ref["grad"], (ref["count"] + 3)[:, None] * U * ref["size"])
        assert (o[b - a:] == 3).all()
    # rows outside the slice, and of padding, are not read
    gd[torch.as_tensor((tok < 313) | (tok >= 900)).cuda()] = float("nan")
    assert B.dg_token_embed_backward(gd, i32(tok), 1000, 1.0, vocab_start=313, vocab_end=900).isfinite().all()


def test_gradient_without_positions(B):
    o = empty(9, 5, "bf16", "odd")
    g = torch.empty(0, 5, device="cuda")
    B.dg_token_embed_backward(g, i32([]), 9, 1.0, out=o)
    assert not o.any()
    untouched(o, "bf16")
    o.fill_(2)
    B.dg_token_embed_backward(g, i32([]), 9, 1.0, out=o, accumulate=True)
    assert (o == 2).all()
    assert B.dg_token_embed(torch.ones(4, 5, device="cuda"), i32([])).shape == (0, 5)


# --------------------------------------------------------------------------- norm

def size(rng, R, d):
    return np.exp(rng.normal(size=(R, 1))) * np.where(rng.random((1, d)) < 0.02, 30.0, 1.0) * rng.normal(size=(R, d))


def check_codes(o, ref):
    """Codes and scales against y: each the nearest to y at a scale of the row's largest |y|."""
    s = o["scale"].double().cpu().numpy()
    top = np.abs(ref).max(1)
    close(s, top / 448, 57 * U * top / 448)
    q = e4m3_decode(o["out"].cpu().numpy()) * s[:, None]
    close(q, ref, np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * s[:, None]) * (1 + 4 * U) + 60 * U * np.abs(ref))


WIDTHS = [1, 7, 8, 33, 255, 256, 257, 1153, 2048, 2049, 2816, 4097, 8192, 8200, 16385, 32768]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("x,res,out", [("f32", None, "f32"), ("bf16", "f32", "e4m3"), ("bf16", "bf16", "bf16"),
                                       ("f32", "bf16", "e4m3"), ("f32", "f32", "bf16"), ("bf16", None, "f32")])
@pytest.mark.parametrize("layout", ["wide", "odd"])
def test_norm(B, d, x, res, out, layout):
    rng = np.random.default_rng(d)
    R = 5 if d < 1000 else 3
    offset, wk = (1.0, "bf16") if d % 2 else (0.0, "f32")
    xd, xv = place(size(rng, R, d), x, layout)
    rd, rv = place(size(rng, R, d), res, layout) if res else (None, None)
    wd, wv = place(1 - offset + 0.3 * rng.normal(size=(1, d)), wk, "odd" if layout == "odd" else "dense")
    o = {"out": empty(R, d, out, layout)}
    if res:
        o["hidden"] = empty(R, d, res, layout)
    B.dg_rms_norm(xd, wd[0], residual=rd, eps=1e-5, weight_offset=offset, out=o)
    ref = H.rms_norm(xv, rv, offset + wv, 1e-5)
    close(o["rstd"], ref["rstd"], 52 * U * ref["rstd"])
    if res:
        close(o["hidden"], ref["hidden"], (HALF[res] + U) * np.abs(ref["hidden"]))
        untouched(o["hidden"], res)
    if out == "e4m3":
        check_codes(o, ref["out"])
    else:
        close(o["out"], ref["out"], (56 * U + HALF[out]) * np.abs(ref["out"]))
    untouched(o["out"], out)


def test_norm_without_weight_and_many_rows(B):
    rng = np.random.default_rng(0)
    xd, xv = place(size(rng, 3001, 130), "bf16")
    got = B.dg_rms_norm(xd)
    ref = H.rms_norm(xv, None, 1.0, 1e-6)
    close(got["out"], ref["out"], (56 * U + 2.0 ** -8) * np.abs(ref["out"]))
    assert sorted(got) == ["out", "rstd"] and got["out"].dtype == torch.bfloat16


def test_norm_of_many_rows(B):
    """Several turns of every CTA, of rows that begin on 16-byte boundaries and of others."""
    g = torch.Generator(device="cuda").manual_seed(1)
    R, d = 20011, 264
    x, res, up = (torch.randn(R, d + 8, generator=g, device="cuda") for _ in range(3))
    w = torch.randn(d, generator=g, device="cuda")
    for c in (0, 1):
        v = [t[:, c:c + d] for t in (x, res, up)]
        o = B.dg_rms_norm(v[0], w, residual=v[1], dtype=torch.uint8)
        h = v[0].double() + v[1].double()
        rstd = (h.square().mean(1) + 1e-6) ** -0.5
        y = h * rstd[:, None] * w.double()
        assert ((o["hidden"] - h).abs() <= U * h.abs()).all() and ((o["rstd"] - rstd).abs() <= 52 * U * rstd).all()
        s, top = o["scale"].double()[:, None], y.abs().amax(1, keepdim=True)
        assert ((s - top / 448).abs() <= 57 * U * top / 448).all()
        q = o["out"].view(torch.float8_e4m3fn).double() * s
        assert ((q - y).abs() <= torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s) * (1 + 4 * U) + 60 * U * y.abs()).all()
        b = B.dg_rms_norm_backward(v[2], o["hidden"], o["rstd"], w, grad_hidden=v[0])
        h, rs, gw = o["hidden"].double(), o["rstd"].double()[:, None], v[2].double() * w.double()
        xh = h * rs
        inner, size = (gw * xh).mean(1, keepdim=True), (gw * xh).abs().mean(1, keepdim=True)
        ref = v[0].double() + rs * (gw - xh * inner)
        tol = rs * (6 * U * gw.abs() + 102 * U * xh.abs() * size) + 4 * U * ref.abs() + U * v[0].abs()
        assert ((b["grad"] - ref).abs() <= tol).all()
        terms = v[2].double() * xh
        assert ((b["grad_weight"] - terms.sum(0)).abs() <= (R + 3) * U * terms.abs().sum(0)).all()


def test_norm_hidden_of_its_own_type(B):
    rng = np.random.default_rng(6)
    xd, xv = place(size(rng, 30, 520), "f32")
    rd, rv = place(size(rng, 30, 520), "bf16")
    ref = B.dg_rms_norm(xd, residual=rd)
    for kind in ("f32", "bf16"):
        for res, h in ((rd, xv + rv), (None, xv)):
            o = B.dg_rms_norm(xd, residual=res, out={"hidden": empty(30, 520, kind)})
            close(o["hidden"], h, (HALF[kind] + U) * np.abs(h))
            untouched(o["hidden"], kind)
        close(B.dg_rms_norm(xd, residual=rd, out={"hidden": empty(30, 520, kind)})["out"], np64(ref["out"]),
              56 * U * np.abs(np64(ref["out"])))
    o = B.dg_rms_norm(xd, residual=rd, out={"hidden": None})
    assert o["hidden"] is None and torch.equal(o["out"], ref["out"])


def np64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("out", ["f32", "e4m3"])
def test_rows_of_zeros_and_of_what_is_no_number(B, out):
    x = torch.ones(6, 300, device="cuda")
    x[1] = 0
    x[2, 7], x[3, 299], x[4, 0] = float("nan"), float("inf"), -float("inf")
    x[5] = 1e-30
    o = B.dg_rms_norm(x, dtype=T[out])
    # a row of zeros stays one, and rows do not reach into one another
    assert not o["out"][1].any() and float(o["rstd"][1]) == pytest.approx(1e3, rel=1e-6)
    assert float(o["rstd"][0]) == pytest.approx(1.0, rel=1e-6)
    if out == "e4m3":
        assert o["scale"][1] == 0 and (o["out"][0] == 0x7E).all()
        assert not o["scale"][2:5].isfinite().any() and float(o["scale"][5]) == pytest.approx(1e-27 / 448, rel=1e-5)
        assert (o["out"][5] == 0x7E).all()
    else:
        assert not o["out"][2].isfinite().any() and not o["out"][3, 299].isfinite() and not o["out"][4, 0].isfinite()
        assert o["out"][[0, 1, 5]].isfinite().all()
    z = B.dg_rms_norm(torch.zeros(2, 9, device="cuda"), eps=0.0, dtype=T["e4m3"])["scale"]
    assert z.isnan().all()                                   # 0 / 0: no direction


def test_norm_in_place(B):
    rng = np.random.default_rng(2)
    xd, xv = place(size(rng, 40, 999), "f32")
    rd, rv = place(size(rng, 40, 999), "f32")
    w = f32(rng.normal(size=999))
    ref = B.dg_rms_norm(xd, w, residual=rd)
    x2, r2 = xd.clone(), rd.clone()
    x2, _ = place(xv, "f32")
    r2, _ = place(rv, "f32")
    B.dg_rms_norm(x2, w, residual=r2, out={"out": x2, "hidden": r2})
    assert torch.equal(x2, ref["out"]) and torch.equal(r2, ref["hidden"])
    x2, _ = place(xv, "f32")
    r2, _ = place(rv, "f32")
    B.dg_rms_norm(x2, w, residual=r2, out={"out": r2, "hidden": x2})
    assert torch.equal(r2, ref["out"]) and torch.equal(x2, ref["hidden"])
    with pytest.raises(B.DgError, match="overlaps"):
        B.dg_rms_norm(xd, w, residual=rd, out={"out": ref["out"], "hidden": ref["out"]})


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("g,h,up", [("f32", "f32", None), ("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"),
                                    ("f32", "bf16", "f32"), ("bf16", "f32", "bf16")])
@pytest.mark.parametrize("layout", ["wide", "odd"])
def test_norm_gradient(B, d, g, h, up, layout):
    rng = np.random.default_rng(d)
    R = 700 if d < 100 else 37 if d < 3000 else 5
    offset, wk = (1.0, "bf16") if d % 2 else (0.0, "f32")
    hd, hv = place(size(rng, R, d), h, layout)
    gd, gv = place(rng.normal(size=(R, d)), g, layout)
    ud, uv = place(rng.normal(size=(R, d)), up, layout) if up else (None, None)
    wd, wv = place(1 - offset + 0.3 * rng.normal(size=(1, d)), wk, "odd" if layout == "odd" else "dense")
    rstd = f32((np.mean(hv * hv, 1) + 1e-6) ** -0.5)
    rs = rstd.double().cpu().numpy()[:, None]
    o = {"grad": empty(R, d, h, layout)}
    B.dg_rms_norm_backward(gd, hd, rstd, wd[0], offset, grad_hidden=ud, out=o)
    w = offset + wv
    ref = H.rms_norm_backward(gv, hv, rs[:, 0], w, uv)
    t1, xh = np.abs(gv * w), np.abs(hv * rs)
    inner = np.mean(t1 * xh, 1, keepdims=True)
    tol = rs * (6 * U * t1 + (96 + 6) * U * xh * inner) + 2 * U * np.abs(ref["grad"]) + HALF[h] * np.abs(ref["grad"])
    if up:
        tol = tol + U * np.abs(uv)
    close(o["grad"], ref["grad"], tol)
    untouched(o["grad"], h)
    terms = np.sum(np.abs(gv) * xh, axis=0)
    close(o["grad_weight"], ref["grad_weight"], (R + 3) * U * terms + HALF[wk] * np.abs(ref["grad_weight"]))
    again = B.dg_rms_norm_backward(gd, hd, rstd, wd[0], offset, grad_hidden=ud)
    assert torch.equal(again["grad"], o["grad"]) and torch.equal(again["grad_weight"], o["grad_weight"])


def test_norm_gradient_in_place_and_partial(B):
    rng = np.random.default_rng(5)
    g, h, up = (f32(rng.normal(size=(50, 264))) for _ in range(3))
    w, rstd = f32(rng.normal(size=264)), f32(rng.uniform(0.5, 2, 50))
    ref = B.dg_rms_norm_backward(g, h, rstd, w, grad_hidden=up)
    for k in range(3):
        three = [t.clone() for t in (g, h, up)]
        o = B.dg_rms_norm_backward(three[0], three[1], rstd, w, grad_hidden=three[2], out={"grad": three[k]})
        assert o["grad"] is three[k] and torch.equal(o["grad"], ref["grad"])
        assert torch.equal(o["grad_weight"], ref["grad_weight"])
    o = B.dg_rms_norm_backward(g, h, rstd, w, grad_hidden=up, out={"grad_weight": None})
    assert torch.equal(o["grad"], ref["grad"]) and o["grad_weight"] is None
    o = B.dg_rms_norm_backward(g, h, rstd)
    close(o["grad"], H.rms_norm_backward(*(t.double().cpu().numpy() for t in (g, h, rstd)), 1.0)["grad"], 1e-4)
    o = B.dg_rms_norm_backward(g[:0], h[:0], rstd[:0], w)
    assert o["grad"].shape == (0, 264) and not o["grad_weight"].any()


# --------------------------------------------------------------------------- head

def check_head(B, R, V, d, out, pad=0, seed=0, zero=False):
    rng = np.random.default_rng(R + V + d + seed)
    finite = np.delete(np.arange(256), [0x7F, 0xFF])

    def codes(n):
        # what lies in the columns past d is NaN
        buf = torch.full((n, (d + 15) // 16 * 16 + 16 * pad), 0x7F, dtype=torch.uint8, device="cuda")
        c = rng.choice(finite, (n, d)).astype(np.uint8)
        buf[:, :d] = torch.as_tensor(c).cuda()
        return buf[:, :d], e4m3_decode(c)
    X, x = codes(R)
    Q, q = codes(V)
    xs, s = rng.uniform(0.5, 2, R).astype(np.float32), rng.uniform(1e-3, 2e-3, V).astype(np.float32)
    if zero:
        xs[0], s[-1] = 0, 0
    o = empty(R, V, out)
    B.dg_head_e4m3(X, f32(xs), Q, f32(s), out=o)
    ref, terms = H.head(x, xs, q, s), H.head(np.abs(x), xs, np.abs(q), s)
    close(o, ref, (d / 32 + 33) * 2.0 ** -23 * terms + (3 * U + HALF[out]) * np.abs(ref))
    untouched(o, out)
    return o


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("R,V,d", [(1, 1, 1), (1, 1000, 128), (2, 127, 31), (31, 129, 32), (32, 255, 33), (33, 256, 127),
                                   (64, 257, 129), (100, 513, 160), (129, 640, 255), (255, 100, 384), (256, 1000, 511),
                                   (257, 300, 64), (300, 511, 700), (513, 700, 96), (700, 260, 2817)])
def test_head(B, R, V, d, out):
    check_head(B, R, V, d, out, pad=R % 2)


@pytest.mark.parametrize("R,V,d", [(1, 120003, 48), (40, 70001, 80), (300, 50001, 16), (1030, 9999, 40)])
def test_head_over_many_tiles(B, R, V, d):
    check_head(B, R, V, d, "f32", zero=True)
    check_head(B, R, V, d, "bf16", seed=1)


def test_head_twice(B):
    a = check_head(B, 200, 3001, 2816, "f32")
    assert torch.equal(a, check_head(B, 200, 3001, 2816, "f32"))


def test_head_of_codes_that_are_no_number(B):
    X = torch.zeros(3, 64, dtype=torch.uint8, device="cuda")
    Q = torch.full((300, 64), 0x38, dtype=torch.uint8, device="cuda")
    X[1, 5], Q[17, 0] = 0x7F, 0xFF
    o = B.dg_head_e4m3(X, torch.ones(3, device="cuda"), Q, torch.ones(300, device="cuda"))
    nan = torch.zeros(3, 300, dtype=torch.bool, device="cuda")
    nan[1], nan[:, 17] = True, True
    assert torch.equal(o.isnan(), nan) and not o[~nan].any()
