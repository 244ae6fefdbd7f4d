"""The hidden stream's calls together: with the sampler's loop, in autograd, in captured graphs, on streams.

Tolerances as in test_gpu_hidden.py, of which this takes the ones of the operators that it runs together."""
import numpy as np
import pytest
import torch

from denoising_sampler_step_gb300 import inputs
from oracle import e4m3_decode, hidden_oracle as H
from test_gpu_hidden import B, close, device_status_stays_clear, f32, i32  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def np64(t):
    return t.double().cpu().numpy()


@pytest.fixture(params=["bf16", "e4m3"])
def ends(request, B):
    """(TiedEnds, loop, canvas, budgets) of two canvases of the tiny workload."""
    from denoising_sampler_step_gb300.step import SamplerLoop, TiedEnds
    wl = inputs.WORKLOADS["tiny"]
    n, R = 2, 2 * wl.L_c
    g = torch.Generator(device="cuda").manual_seed(5)
    W = (torch.randn(wl.V, wl.d, generator=g, device="cuda") / wl.d ** 0.5).bfloat16()
    kw = {}
    if request.param == "e4m3":
        W, kw["scale"] = B.dg_quantize_e4m3(W)
    w_in, w_out = (0.1 * torch.randn(wl.d, generator=g, device="cuda") for _ in range(2))
    e = TiedEnds(W, R, wl.gamma, w_in, w_out, weight_offset=1.0, **kw)
    loop = SamplerLoop(W, n, wl.L_c, wl.V, wl.gamma, stable_steps=2, entropy_threshold=0.5, step_limit=8, **kw)
    canvas = torch.randint(wl.V, (R,), generator=g, device="cuda").int()
    return e, loop, canvas, torch.full((n,), 20.0, device="cuda")


def denoise(e, loop, canvas, budgets, steps, seen=None):
    """A loop whose model is the identity: the first norm's output is the last layer's."""
    loop.reset(canvas)
    loop.out["E"].zero_()
    for _ in range(steps):
        h, y = e.inputs(loop.state["canvas"], loop.out["E"])
        x = e.logits(y, residual=h)
        if seen is not None:
            seen.append({k: v.clone() for k, v in dict(canvas=loop.state["canvas"], E=loop.out["E"], x=e.embedded, h=h,
                                                       y=y, rstd=e.first["rstd"], q=e.last["out"],
                                                       s=e.last["scale"], logits=x).items()})
        loop(x, budgets)
    return {**{k: v.clone() for k, v in loop.state.items()}, **{k: v.clone() for k, v in loop.out.items()}}


def test_a_denoising_loop_with_both_ends(B, ends):
    e, loop, canvas, budgets = ends
    seen = []
    denoise(e, loop, canvas, budgets, 3, seen)
    W = np64(e.W) if e.w_scale is None else e4m3_decode(e.Q.cpu().numpy()) * np64(e.scale)[:, None]
    Q = e4m3_decode(e.Q.cpu().numpy())
    # (a model that is the identity names its own tokens; what changes from step to step is E)
    assert not seen[0]["E"].any() and seen[1]["E"].any() and not torch.equal(seen[0]["logits"], seen[1]["logits"])
    for o in seen:
        ref = H.token_embed(W, o["canvas"].cpu().numpy(), e.gamma)
        close(o["x"], ref, (3 * U + 2.0 ** -8) * np.abs(ref))
        n1 = H.rms_norm(np64(o["x"]), np64(o["E"]), 1 + np64(e.norm_in), e.eps)
        close(o["h"], n1["hidden"], 2 * U * np.abs(n1["hidden"]))
        close(o["y"], n1["out"], (56 * U + 2.0 ** -8) * np.abs(n1["out"]))
        n2 = H.rms_norm(np64(o["y"]), np64(o["h"]), 1 + np64(e.norm_out), e.eps)["out"]
        q = e4m3_decode(o["q"].cpu().numpy())
        s = np64(o["s"])
        close(q * s[:, None], n2, np.maximum(2.0 ** -4 * np.abs(n2), 2.0 ** -10 * s[:, None]) * (1 + 4 * U) + 60 * U * np.abs(n2))
        terms = H.head(np.abs(q), s, np.abs(Q), np64(e.scale))
        ref = H.head(q, s, Q, np64(e.scale))
        close(o["logits"], ref, (q.shape[1] / 32 + 33) * 2.0 ** -23 * terms + 4 * U * np.abs(ref))


def test_the_loop_captured_and_replayed(B, ends):
    e, loop, canvas, budgets = ends
    ref = denoise(e, loop, canvas, budgets, 4)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            h, y = e.inputs(loop.state["canvas"], loop.out["E"])
            loop(e.logits(y, residual=h), budgets)
        for _ in range(2):
            loop.reset(canvas)
            loop.out["E"].zero_()
            for _ in range(4):
                graph.replay()
            s.synchronize()
            for k, v in ref.items():
                got = loop.state.get(k, loop.out.get(k))
                assert torch.equal(got, v), k


def everything(B, g, stream=None):
    """Calls of all operators on inputs of generator g, in a closure, with what they write."""
    R, V, d = 3000, 5000, 264
    W = torch.randn(V, d, generator=g, device="cuda").bfloat16()
    Q, scale = B.dg_quantize_e4m3(W)
    tok = torch.randint(V, (R,), generator=g, device="cuda").int()
    tok[torch.rand(R, generator=g, device="cuda") < 0.4] = 7
    res = torch.randn(R, d, generator=g, device="cuda")
    w = torch.randn(d, generator=g, device="cuda")
    ws, nws = B.embed_workspace(R, V, d, "cuda"), B.norm_workspace(R, d, "cuda")
    o = {"x": torch.empty(R, d, dtype=torch.bfloat16, device="cuda"), "table": torch.empty(V, d, device="cuda"),
         "logits": torch.empty(64, V, device="cuda"),
         "n": {"out": torch.empty(R, 272, dtype=torch.uint8, device="cuda")[:, :d], "scale": torch.empty(R, device="cuda"),
               "rstd": torch.empty(R, device="cuda"), "hidden": torch.empty(R, d, device="cuda")},
         "b": {"grad": torch.empty(R, d, device="cuda"), "grad_weight": torch.empty(d, device="cuda")}}

    def run():
        B.dg_token_embed(W, tok, 2.0, out=o["x"], stream=stream)
        B.dg_rms_norm(o["x"], w, residual=res, out=o["n"], stream=stream)
        B.dg_head_e4m3(o["n"]["out"][:64], o["n"]["scale"][:64], Q, scale, out=o["logits"], stream=stream)
        B.dg_rms_norm_backward(res, o["n"]["hidden"], o["n"]["rstd"], w, out=o["b"], ws=nws, stream=stream)
        B.dg_token_embed_backward(o["b"]["grad"], tok, V, 2.0, out=o["table"], ws=ws, stream=stream)

    def flat():
        return [t.clone() for t in (o["x"], o["table"], o["logits"], *o["n"].values(), *o["b"].values())]
    return run, flat


def test_on_two_streams_at_once(B):
    ref = []
    for seed in (1, 2):
        run, flat = everything(B, torch.Generator(device="cuda").manual_seed(seed))
        run()
        ref.append(flat())
    streams = [torch.cuda.Stream() for _ in range(2)]
    pairs = [everything(B, torch.Generator(device="cuda").manual_seed(seed), s) for seed, s in zip((1, 2), streams)]
    torch.cuda.synchronize()
    for _ in range(10):
        for run, _ in pairs:
            run()
    torch.cuda.synchronize()
    for (_, flat), r in zip(pairs, ref):
        for a, b in zip(flat(), r):
            assert torch.equal(a, b)


def test_captured_and_replayed(B):
    run, flat = everything(B, torch.Generator(device="cuda").manual_seed(3))
    run()
    ref = flat()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
        run()
    for _ in range(3):
        graph.replay()
    for a, b in zip(flat(), ref):
        assert torch.equal(a, b)


def test_what_the_binding_refuses(B, monkeypatch):
    x, tok = torch.zeros(4, 16, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    codes = torch.zeros(4, 16, dtype=torch.uint8, device="cuda")
    one = torch.ones(4, device="cuda")
    calls = [lambda: B.dg_token_embed(x, tok), lambda: B.dg_token_embed_backward(x, tok, 9), lambda: B.dg_rms_norm(x),
             lambda: B.dg_rms_norm_backward(x, x, one), lambda: B.dg_head_e4m3(codes, one, codes, one)]
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_cuda_getDevice", lambda: 1)     # (one GPU here: as if the second were current)
        for call in calls:
            with pytest.raises(ValueError, match="current device"):
                call()
    for call in calls:
        call()
    for bad, err in [(lambda: B.dg_token_embed(x, tok.long()), ValueError), (lambda: B.dg_token_embed(x.half(), tok), TypeError),
                     (lambda: B.dg_token_embed(x, tok[::2]), ValueError), (lambda: B.dg_token_embed(x.t(), tok), ValueError),
                     (lambda: B.dg_token_embed(codes, tok), B.DgError), (lambda: B.dg_token_embed(x, tok, scale=one), B.DgError),
                     (lambda: B.dg_token_embed(x, tok, out=x), B.DgError), (lambda: B.dg_token_embed(x, tok.cpu()), ValueError),
                     (lambda: B.dg_token_embed(x, tok, vocab_start=2, vocab_end=9, V=9), B.DgError),
                     (lambda: B.dg_token_embed_backward(x, tok, 9, accumulate=True), ValueError),
                     (lambda: B.dg_token_embed_backward(x[:1].expand(4, 16), tok, 9), B.DgError),
                     (lambda: B.dg_token_embed_backward(x, tok, 9, out=torch.zeros(8, 16, device="cuda")), B.DgError),
                     (lambda: B.dg_rms_norm(x, one), ValueError), (lambda: B.dg_rms_norm(x, residual=x[:, :8]), ValueError),
                     (lambda: B.dg_rms_norm(x, x[0].half()), B.DgError), (lambda: B.dg_rms_norm(x, eps=-1.0), B.DgError),
                     (lambda: B.dg_rms_norm_backward(x, x.bfloat16(), one, out={"grad": torch.zeros_like(x)}), TypeError),
                     (lambda: B.dg_rms_norm_backward(x, x, one, out={"grad_weight": one}), ValueError),
                     (lambda: B.dg_head_e4m3(x, one, codes, one), TypeError),
                     (lambda: B.dg_head_e4m3(codes, one, codes[:, :8], one), ValueError),
                     (lambda: B.dg_head_e4m3(codes[:, 1:], one, codes[:, 1:], one), B.DgError),
                     (lambda: B.dg_head_e4m3(codes, one[:3], codes, one), ValueError)]:
        with pytest.raises(err):
            bad()


# --------------------------------------------------------------------------- autograd

@pytest.fixture(scope="module")
def T(B):
    from denoising_sampler_step_gb300 import training
    return training


def plain_norm(x, w, res, eps, offset):
    h = x if res is None else x + res
    return h * (h.square().mean(1, keepdim=True) + eps) ** -0.5 * (offset + w), h


@pytest.mark.parametrize("res", [True, False])
def test_gradients_through_lookup_and_norm(T, res):
    g = torch.Generator(device="cuda").manual_seed(1)
    R, V, d = 90, 40, 100
    table = torch.randn(V, d, generator=g, device="cuda").requires_grad_(True)
    w = torch.randn(d, generator=g, device="cuda").requires_grad_(True)
    r = torch.randn(R, d, generator=g, device="cuda").requires_grad_(True) if res else None
    tok = torch.randint(V, (R,), generator=g, device="cuda").int()
    tok[::7] = -1
    up, uh = (torch.randn(R, d, generator=g, device="cuda") for _ in range(2))
    leaves = [table, w] + ([r] if res else [])

    def mine(table, w, r=None):
        y, h = T.rms_norm(T.token_embed(table, tok, 3.0), w, residual=r, eps=1e-3, weight_offset=1.0)
        return (y * up).sum() + (0 if h is None else (h * uh).sum())

    def plain(table, w, r=None):
        x = torch.where(tok[:, None] >= 0, 3.0 * table[tok.clamp(min=0).long()], 0)
        y, h = plain_norm(x, w, r, 1e-3, 1.0)
        return (y * up.double()).sum() + (0 if r is None else (h * uh.double()).sum())
    got = torch.autograd.grad(mine(*leaves), leaves)
    wide = [t.detach().double().requires_grad_(True) for t in leaves]
    ref = torch.autograd.grad(plain(*wide), wide)
    for a, b in zip(got, ref):
        # a row of zeros (padding without a residual) has rstd 1e1.5; sums of up to 90 terms of a few units each
        assert (a - b).abs().max() <= 2e-5 * max(1.0, float(b.abs().max()))
    # and differences of the fp64 expression along random directions
    for k, t in enumerate(wide):
        v = torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64)
        with torch.no_grad():
            two = [plain(*[u + s * 1e-5 * v if i == k else u for i, u in enumerate(wide)]) for s in (1, -1)]
        slope = float(two[0] - two[1]) / 2e-5
        assert abs(slope - float((got[k] * v).sum())) <= 1e-4 * float((got[k].abs() * v.abs()).sum())


def test_types_of_gradients(T):
    x = torch.randn(6, 40, device="cuda").bfloat16().requires_grad_(True)
    r = torch.randn(6, 40, device="cuda").requires_grad_(True)
    w = torch.ones(40, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y, h = T.rms_norm(x, w, residual=r)
    assert y.dtype == torch.bfloat16 and h.dtype == torch.float32
    y.float().sum().backward()                              # an expanded upstream gradient, and none for h
    assert x.grad.dtype == torch.bfloat16 and r.grad.dtype == torch.float32 and w.grad.dtype == torch.bfloat16
    x.grad = None
    T.rms_norm(x, w, residual=r)[1].sum().backward()        # y not used at all: h = x + r
    assert (x.grad == 1).all()
    table = torch.randn(9, 40, device="cuda").bfloat16().requires_grad_(True)
    T.token_embed(table, torch.zeros(3, dtype=torch.int32, device="cuda"), 2.0, dtype=torch.float32).sum().backward()
    assert table.grad.dtype == torch.bfloat16 and (table.grad[0] == 6).all() and not table.grad[1:].any()
    with pytest.raises(RuntimeError, match="first derivatives"):
        torch.autograd.grad(T.rms_norm(x, w)[0].sum(), x, create_graph=True)


def test_a_training_step_captured(T):
    """Forward and backward pass in one graph, its gradients those of the eager pass."""
    g = torch.Generator(device="cuda").manual_seed(2)
    tok = torch.randint(50, (64,), generator=g, device="cuda").int()
    res = torch.randn(64, 72, generator=g, device="cuda")
    first = torch.randn(50, 72, generator=g, device="cuda")
    static = first.clone().requires_grad_(True)
    w = torch.ones(72, device="cuda", requires_grad=True)

    def step(table):
        y, h = T.rms_norm(T.token_embed(table, tok, 2.0), w, residual=res)
        return torch.autograd.grad((y * h).sum(), (table, w))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(static)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(static)
    for k in range(2):
        with torch.no_grad():
            static.copy_(first * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        for a, b in zip(kept, step((first * (k + 1)).requires_grad_(True))):
            assert torch.equal(a, b)


def test_the_denoising_run(T):
    from denoising_sampler_step_gb300 import finetune
    lines = []
    r = finetune.denoise(steps=5, log=lines.append)
    assert len(lines) == 1 and np.isfinite(r["denoise"]).all()
