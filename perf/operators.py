"""The training-side operators over the sampler's logits, as cases to be timed and compared.

Four operators work on rows of full-vocabulary logits (fp32 or bf16, a leading dimension that
may exceed V):

* topk        the K largest logits of each row (ties: lowest index), with the tempered
              log-sum-exp: a teacher's top logits, or one position's alternatives when serving;
* distill     the distillation loss from a teacher's top logits, and its gradient;
* policy      the clipped policy loss with a KL term, and its gradient;
* preference  the loss on paired log ratios of packed sequences, and its gradient.

A case's "pass" says which direction one run() takes: "forward" (losses only), "step" (losses
and the gradient of the logits in one call) or "backward" (the gradient from what a forward
call saved).  `own` selects the framework's calls; otherwise the operators run in a plain form
of elementary torch operations in fp32.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one position's top alternatives while serving: the smallest call, latency counts
        dict(name="topk one position", op="topk", R=1, V=262144, K=32, dtype="f32", T=1.0, lse=True),
        # a teacher's pass over one 256-position canvas, its top logits kept for distillation
        dict(name="topk canvas", op="topk", R=256, V=262144, K=64, dtype="f32", T=2.0, lse=True),
        # a bf16 teacher with a ragged vocabulary and a wide K; bf16 has many ties
        dict(name="topk ragged", op="topk", R=1000, V=50001, K=200, dtype="bf16", T=1.0, lse=False),
        # the tiny configuration's 16 positions: launch latency
        dict(name="distill tiny", op="distill", R=16, V=4096, K=16, dtype="f32", T=1.0, tail=False,
             masked=0.0, **{"pass": "step"}),
        # one canvas in the training type, a temperature, the rest of the vocabulary as a bucket
        dict(name="distill canvas", op="distill", R=256, V=262144, K=64, dtype="bf16", T=1.25, tail=True,
             masked=0.0, **{"pass": "step"}),
        # eight canvases, a quarter of the positions masked (prompt or padding): the largest
        dict(name="distill batch", op="distill", R=2048, V=262144, K=128, dtype="f32", T=1.0, tail=False,
             masked=0.25, **{"pass": "step"}),
        # the autograd form: the gradient from the saved log-sum-exp, odd sizes throughout
        dict(name="distill backward", op="distill", R=777, V=100003, K=33, dtype="f32", T=1.5, tail=True,
             masked=0.1, **{"pass": "backward"}),
        # the tiny configuration's 16 positions: launch latency
        dict(name="policy tiny", op="policy", R=16, V=4096, dtype="f32", T=1.0, masked=0.0, **{"pass": "step"}),
        # one canvas of drawn tokens
        dict(name="policy canvas", op="policy", R=256, V=262144, dtype="f32", T=1.0, masked=0.0,
             **{"pass": "step"}),
        # eight canvases in the training type, a quarter of the positions masked
        dict(name="policy batch", op="policy", R=2048, V=262144, dtype="bf16", T=1.0, masked=0.25,
             **{"pass": "step"}),
        # a few short packed sequences of odd lengths, a ragged vocabulary
        dict(name="preference ragged", op="preference", P=3, L=61, V=32003, dtype="bf16", T=1.0, masked=0.0,
             **{"pass": "step"}),
        # four pairs of answers of up to one canvas each
        dict(name="preference canvas", op="preference", P=4, L=256, V=262144, dtype="bf16", T=1.0, masked=0.1,
             **{"pass": "step"}),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["topk", "distill", "policy", "preference"])
    V = _log_int(rng, 1000, 262144)
    R = _log_int(rng, 1, 2048)
    dtype = rng.choice(["f32", "bf16"])
    T = rng.choice([1.0, round(rng.uniform(0.6, 1.6), 2)])
    masked = rng.choice([0.0, round(rng.uniform(0.05, 0.6), 2)])
    if op == "topk":
        return dict(op=op, R=R, V=V, K=_log_int(rng, 1, 512), dtype=dtype, T=T, lse=rng.random() < 0.5)
    if op == "distill":
        return {**dict(op=op, R=R, V=V, K=_log_int(rng, 1, 512), dtype=dtype, T=T, tail=rng.random() < 0.5,
                       masked=masked), "pass": rng.choice(["forward", "step", "step", "backward"])}
    if op == "policy":
        return {**dict(op=op, R=R, V=V, dtype=dtype, T=T, masked=masked),
                "pass": rng.choice(["forward", "step", "step", "backward"])}
    P = _log_int(rng, 1, 16)
    return {**dict(op=op, P=P, L=_log_int(rng, 1, 1024 // P), V=V, dtype=dtype, T=T, masked=masked),
            "pass": rng.choice(["forward", "step", "step"])}


def _lengths(case):
    """Lengths of the 2P packed sequences, fixed by the case: 1 to L, the first one L."""
    r = random.Random(1000 * case["P"] + case["L"])
    return [case["L"]] + [r.randint(1, case["L"]) for _ in range(2 * case["P"] - 1)]


def _rows(case):
    return sum(_lengths(case)) if case["op"] == "preference" else case["R"]


def _masked_rows(case):
    return int(case.get("masked", 0.0) * _rows(case))


# --------------------------------------------------------------------------- inputs

CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.04
BETA, SMOOTHING = 0.1, 0.05


def _logits(g, R, V, dtype):
    """Rows l = s z + bump like the sampler's workloads (s in [0.5, 4], a bump of up to 8 at one
    entry), in storage whose rows start on 16-byte boundaries."""
    x = torch.randn(R, V, generator=g, device="cuda")
    x.mul_(0.5 + 3.5 * torch.rand(R, 1, generator=g, device="cuda"))
    at = torch.randint(V, (R, 1), generator=g, device="cuda")
    x.scatter_add_(1, at, 8.0 * torch.rand(R, 1, generator=g, device="cuda"))
    return _padded(x, dtype)


def _padded(x, dtype):
    R, V = x.shape
    per = 16 // SIZE[dtype]
    buf = torch.zeros(R, (V + per - 1) // per * per, dtype=DTYPES[dtype], device="cuda")
    buf[:, :V] = x
    return buf[:, :V]


def _mask(g, R, n):
    """Row weights of a mean over the rows that count: `n` of them zero."""
    w = torch.full((R,), 1.0 / max(1, R - n), device="cuda")
    w[torch.randperm(R, generator=g, device="cuda")[:n]] = 0.0
    return w


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    R, V, dtype, T = _rows(case), case["V"], case["dtype"], case["T"]
    s = {"case": case, "logits": _logits(g, R, V, dtype)}
    f32 = dict(dtype=torch.float32, device="cuda")
    out = {}
    if case["op"] == "topk":
        K = min(case["K"], V)
        out["values"] = torch.empty(R, K, **f32)
        out["indices"] = torch.empty(R, K, dtype=torch.int32, device="cuda")
        if case["lse"]:
            out["lse"] = torch.empty(R, **f32)
        s["out"] = out
        return s
    s["weight"] = _mask(g, R, _masked_rows(case))
    out["lse"] = torch.empty(R, **f32)
    if case["pass"] != "forward":
        out["grad"] = _padded(torch.zeros(R, V, **f32), dtype)
    if case["op"] == "distill":
        # the teacher: the student's logits moved by noise (a divergence of some tenths of a nat,
        # as while training), of which the top K are kept
        t = s["logits"].float() * 0.8
        t += 1.5 * torch.randn(R, V, generator=g, device="cuda")
        s["teacher"], idx = t.topk(min(case["K"], V), dim=1)
        s["indices"] = idx.to(torch.int32)
        s["teacher_lse"] = (t / T).logsumexp(1) if case["tail"] else None
        del t
        out["loss"] = torch.empty(R, **f32)
        out["tail_logp"] = torch.empty(R, **f32)
        if case["pass"] == "backward":
            z = s["logits"].float() / T
            s["lse"] = z.logsumexp(1)
            z.scatter_(1, idx, -math.inf)
            s["tail_logp"] = z.logsumexp(1) - s["lse"]
            del z
    else:
        # tokens drawn from the policy, and its log-probabilities
        z = s["logits"].float() / T
        lse = z.logsumexp(1)
        gumbel = torch.empty_like(z).exponential_(generator=g).log_().neg_()
        tok = gumbel.add_(z).argmax(1, keepdim=True)
        del gumbel
        logp = z.gather(1, tok)[:, 0] - lse
        del z
        s["token"] = tok[:, 0].to(torch.int32)
        out["logp"] = torch.empty(R, **f32)
        noise = torch.randn(R, generator=g, device="cuda").abs()
        if case["op"] == "policy":
            # the reference lies some tenths of a nat off, to either side
            side = 1.0 - 2.0 * torch.randint(2, (R,), generator=g, device="cuda")
            s["ref_logp"] = logp + side * (0.2 + 0.2 * noise)
            # ratios spread over and past the clipping range, none within 2e-3 of its ends, where
            # the derivative jumps and fp32 rounding would decide
            ratio = torch.exp(0.2 * torch.randn(R, generator=g, device="cuda"))
            for edge in (1.0 - CLIP_LOW, 1.0 + CLIP_HIGH):
                near = (ratio - edge).abs() < 2e-3
                ratio = torch.where(near, torch.full_like(ratio, edge + 4e-3), ratio)
            s["old_logp"] = logp - ratio.log()
            s["advantage"] = torch.randn(R, generator=g, device="cuda")
            if case["pass"] == "backward":
                s["lse"], s["dlogp"] = lse, torch.randn(R, generator=g, device="cuda")
            for k in ("loss", "kl", "dlogp"):
                out[k] = torch.empty(R, **f32)
            out["clipped"] = torch.empty(R, dtype=torch.uint8, device="cuda")
        else:
            # every sequence has become likelier or less likely than under the reference
            lengths = _lengths(case)
            start = np.concatenate([[0], np.cumsum(lengths)])
            s["seq_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
            side = 1.0 - 2.0 * torch.randint(2, (len(lengths),), generator=g, device="cuda")
            side = side.repeat_interleave(torch.tensor(lengths, device="cuda"))
            s["ref_logp"] = logp + side * (0.04 + 0.08 * noise)
            s["weight"] = (s["weight"] > 0).float()
            out["loss"] = torch.empty(case["P"], **f32)
            out["log_ratio"] = torch.empty(2 * case["P"], **f32)
            out["dlogp"] = torch.empty(R, **f32)
    s["out"] = out
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "topk":
        return _plain_topk(s, c)
    return {"distill": _plain_distill, "policy": _plain_policy, "preference": _plain_preference}[c["op"]](s, c)


def _run_own(s, c):
    from denoising_sampler_step_gb300 import binding as B

    x, out, T = s["logits"], s["out"], c["T"]
    if c["op"] == "topk":
        if "ws" not in s:
            s["ws"] = B.topk_workspace(x.shape[0], x.shape[1], out["values"].shape[1], x.device, x.dtype)
        return B.dg_row_topk(x, out["values"].shape[1], temperature=T, ws=s["ws"], out=out)
    if c["op"] == "distill":
        if c["pass"] == "backward":
            return {"grad": B.dg_distill_loss_backward(x, s["indices"], s["teacher"], s["lse"], s["weight"],
                                                       teacher_lse=s["teacher_lse"],
                                                       tail_logp=s["tail_logp"] if c["tail"] else None,
                                                       temperature=T, out=out["grad"])}
        o = B.dg_distill_loss(x, s["indices"], s["teacher"], teacher_lse=s["teacher_lse"], temperature=T,
                              weight=s["weight"], out=out)
        return {k: v for k, v in o.items() if c["tail"] or k != "tail_logp"}
    if c["op"] == "policy":
        if c["pass"] == "backward":
            return {"grad": B.dg_token_logp_backward(x, s["token"], s["lse"], s["dlogp"], scale=s["weight"],
                                                     temperature=T, out=out["grad"])}
        return B.dg_policy_loss(x, s["token"], s["old_logp"], s["advantage"], ref_logp=s["ref_logp"],
                                clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=KL_COEF, temperature=T,
                                weight=s["weight"], out=out)
    return B.dg_preference_loss(x, s["token"], s["ref_logp"], s["seq_start"], beta=BETA,
                                label_smoothing=SMOOTHING, temperature=T, weight=s["weight"], out=out)


def _store(grad, dtype):
    return grad if dtype == "f32" else grad.to(DTYPES[dtype])


def _plain_topk(s, c):
    # the entries as integers in the same order (-0 as +0), the index below them: every key differs
    x = s["logits"].float() + 0.0
    K = s["out"]["values"].shape[1]
    bits = x.view(torch.int32)
    bits = bits ^ ((bits >> 31) & 0x7FFFFFFF)
    low = 0xFFFFFFFF - torch.arange(x.shape[1], device=x.device)
    top = ((bits.to(torch.int64) << 32) | low).topk(K, dim=1).values
    idx = 0xFFFFFFFF - (top & 0xFFFFFFFF)
    r = {"values": s["logits"].float().gather(1, idx), "indices": idx.to(torch.int32)}
    if c["lse"]:
        m = x.amax(1, keepdim=True)
        r["lse"] = m[:, 0] / c["T"] + ((x - m) / c["T"]).exp().sum(1).log()
    return r


def _log_softmax(x, T):
    """(z - m, s, lse): the tempered logits below their maximum, their sum of exponentials, the lse."""
    z = x.float() / T
    m = z.amax(1, keepdim=True)
    z = z - m
    ssum = z.exp().sum(1, keepdim=True)
    return z, ssum, (m + ssum.log())[:, 0]


def _plain_distill(s, c):
    T, w, tail = c["T"], s["weight"], c["tail"]
    on, idx = w != 0, s["indices"].long()
    t = s["teacher"] / T
    if tail:
        logq = t - s["teacher_lse"][:, None]
    else:
        t = t - t.amax(1, keepdim=True)
        logq = t - t.exp().sum(1, keepdim=True).log()
    q = logq.exp()
    q0 = (1.0 - q.sum(1)).clamp(min=0.0) if tail else torch.zeros_like(w)
    if c["pass"] == "backward":
        z = s["logits"].float() / T - s["lse"][:, None]
        p, logp0 = z.exp(), s["tail_logp"]
    else:
        z, ssum, lse = _log_softmax(s["logits"], T)
        logp = z.gather(1, idx) - ssum.log()
        kl = (q * (logq - logp)).sum(1)
        p = z.exp() / ssum
        r = {"lse": torch.where(on, lse, 0.0)}
        if tail:
            logp0 = (z.scatter(1, idx, -math.inf).exp().sum(1) / ssum[:, 0]).log()
            kl = kl + torch.where(q0 > 0, q0 * (q0.log() - logp0), 0.0)
            r["tail_logp"] = torch.where(on, logp0, 0.0)
        r["loss"] = torch.where(on, T * T * kl, 0.0)
        if c["pass"] == "forward":
            return r
    mass = (q.sum(1) + q0)[:, None]
    if tail:
        grad = p * (mass - (q0 / logp0.exp())[:, None])
        grad.scatter_(1, idx, p.gather(1, idx) * mass - q)
    else:
        grad = p * mass
        grad.scatter_add_(1, idx, -q)
    grad = _store(grad * (w * T)[:, None], c["dtype"])
    return {"grad": grad} if c["pass"] == "backward" else {**r, "grad": grad}


def _token_grad(p, token, coef, c):
    grad = p * -coef[:, None]
    grad.scatter_add_(1, token[:, None], coef[:, None])
    return _store(grad, c["dtype"])


def _plain_policy(s, c):
    T, w, token = c["T"], s["weight"], s["token"].long()
    if c["pass"] == "backward":
        p = (s["logits"].float() / T - s["lse"][:, None]).exp()
        return {"grad": _token_grad(p, token, s["dlogp"] * w / T, c)}
    on = w != 0
    z, ssum, lse = _log_softmax(s["logits"], T)
    logp = (z.gather(1, token[:, None]) - ssum.log())[:, 0]
    ratio, A = (logp - s["old_logp"]).exp(), s["advantage"]
    raw, cut = ratio * A, ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * A
    d = s["ref_logp"] - logp
    kl = d.expm1() - d
    clipped = raw > cut
    dlogp = torch.where(clipped, 0.0, -raw) + KL_COEF * -d.expm1()
    loss = KL_COEF * kl - torch.minimum(raw, cut)
    r = {"loss": loss, "logp": logp, "lse": lse, "kl": kl, "dlogp": dlogp}
    r = {k: torch.where(on, v, 0.0) for k, v in r.items()}
    r["clipped"] = (clipped & on).to(torch.uint8)
    if c["pass"] == "step":
        r["grad"] = _token_grad(z.exp() / ssum, token, r["dlogp"] * w / T, c)
    return r


def _plain_preference(s, c):
    T, w, token, P = c["T"], s["weight"], s["token"].long(), c["P"]
    on = w != 0
    z, ssum, lse = _log_softmax(s["logits"], T)
    logp = (z.gather(1, token[:, None]) - ssum.log())[:, 0]
    start = s["seq_start"].long()
    seq = torch.bucketize(torch.arange(len(w), device=w.device), start[1:], right=True)
    ratio = torch.zeros(2 * P, device=w.device).index_add(0, seq, w * (logp - s["ref_logp"]))
    zz = BETA * (ratio[0::2] - ratio[1::2])
    # -ln sigmoid(x) = max(-x, 0) + ln(1 + exp(-|x|))
    up, down = [(-v).clamp(min=0.0) + (1.0 + (-v.abs()).exp()).log() for v in (zz, -zz)]
    dz = SMOOTHING / (1.0 + (-zz).exp()) - (1.0 - SMOOTHING) / (1.0 + zz.exp())
    sign = 1.0 - 2.0 * (seq % 2)
    dlogp = BETA * dz[seq // 2] * sign * w
    r = {"loss": (1.0 - SMOOTHING) * up + SMOOTHING * down, "log_ratio": ratio, "dlogp": dlogp,
         "logp": torch.where(on, logp, 0.0), "lse": torch.where(on, lse, 0.0)}
    if c["pass"] == "step":
        r["grad"] = _token_grad(z.exp() / ssum, token, dlogp / T, c)
    return r


# --------------------------------------------------------------------------- cost

def work(case):
    R, V, b = _rows(case), case["V"], SIZE[case["dtype"]]
    if case["op"] == "topk":
        K = min(case["K"], V)
        return {"bytes": R * V * b + R * K * 8 + 4 * R, "flops": (6 if case["lse"] else 1) * R * V}
    live = R - _masked_rows(case)
    rows = 4 * R * {"distill": 4, "policy": 10, "preference": 6}[case["op"]]
    if case["op"] == "distill":
        rows += live * min(case["K"], V) * 8
    if case["pass"] == "forward":
        return {"bytes": live * V * b + rows, "flops": 4 * live * V}
    return {"bytes": (live + R) * V * b + rows, "flops": (4 if case["pass"] == "backward" else 8) * live * V}


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The operators from their definitions in float64, the gradients by differentiating them, a
    block of rows at a time."""
    s = prepare(case, seed)
    out = s.pop("out")
    R, V = s["logits"].shape
    step = max(1, (1 << 24) // V)
    if case["op"] == "topk":
        if not case["lse"]:
            return None
        lse = [(s["logits"][i:i + step].double() / case["T"]).logsumexp(1) for i in range(0, R, step)]
        return {"values": None, "indices": None, "lse": torch.cat(lse)}
    if case["op"] == "preference":
        return _exact_preference(s, case, step)
    got = {}
    for i in range(0, R, step):
        rows = {k: (v[i:i + step].double() if v.is_floating_point() else v[i:i + step].long())
                for k, v in s.items() if isinstance(v, torch.Tensor)}
        x = rows["logits"].requires_grad_(case["pass"] != "forward")
        block = (_exact_distill if case["op"] == "distill" else _exact_policy)(rows, x, case)
        if case["pass"] != "forward":
            total = block.pop("total")
            block["grad"], = torch.autograd.grad(total, x)
            if case["pass"] == "backward":
                block = {"grad": block["grad"]}
        block.pop("total", None)
        for k, v in block.items():
            got.setdefault(k, []).append(v.detach())
    got = {k: torch.cat(v) for k, v in got.items()}
    if case["pass"] != "backward" and case["op"] == "policy":
        got["clipped"] = None
    return got


def _exact_distill(r, x, case):
    T, w = case["T"], r["weight"]
    logp = torch.log_softmax(x / T, 1)
    if case["tail"]:
        q = torch.exp(r["teacher"] / T - r["teacher_lse"][:, None])
        rest = (1.0 - q.sum(1)).clamp(min=0.0)
    else:
        q = torch.softmax(r["teacher"] / T, 1)
    if case["pass"] == "backward":
        # p as the saved values give it: the gradient is linear in it
        p = torch.exp(x.detach() / T - r["lse"][:, None])
        target = torch.zeros_like(p).scatter_(1, r["indices"], q)
        if case["tail"]:
            share = rest / torch.exp(r["tail_logp"])
            inside = torch.zeros_like(p).scatter_(1, r["indices"], 1.0)
            target = target + (1.0 - inside) * p * share[:, None]
            q_all = q.sum(1) + rest
        else:
            q_all = q.sum(1)
        return {"total": (T * w[:, None] * (q_all[:, None] * p - target) * x).sum()}
    loss = torch.special.xlogy(q, q).sum(1) - (q * logp.gather(1, r["indices"])).sum(1)
    got = {"lse": torch.logsumexp(x / T, 1)}
    if case["tail"]:
        got["tail_logp"] = torch.logsumexp(logp.scatter(1, r["indices"], -math.inf), 1)
        loss = loss + torch.special.xlogy(rest, rest) - rest * got["tail_logp"]
    got["loss"] = T * T * loss
    got = {k: torch.where(w != 0, v, 0.0) for k, v in got.items()}
    got["total"] = (w * got["loss"]).sum()
    return got


def _exact_policy(r, x, case):
    T, w = case["T"], r["weight"]
    if case["pass"] == "backward":
        p = torch.exp(x.detach() / T - r["lse"][:, None])
        hot = torch.zeros_like(p).scatter_(1, r["token"][:, None], 1.0)
        return {"total": ((r["dlogp"] * w / T)[:, None] * (hot - p) * x).sum()}
    lse = torch.logsumexp(x / T, 1)
    logp = x.gather(1, r["token"][:, None])[:, 0] / T - lse
    leaf = logp.detach().requires_grad_(True)
    def terms(lp):
        ratio = torch.exp(lp - r["old_logp"])
        gain = torch.minimum(ratio * r["advantage"],
                             torch.clamp(ratio, 1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * r["advantage"])
        back = r["ref_logp"] - lp
        return torch.expm1(back) - back, gain
    kl, gain = terms(leaf)
    dlogp, = torch.autograd.grad((KL_COEF * kl - gain).sum(), leaf)
    kl, gain = terms(logp)
    got = {"loss": KL_COEF * kl - gain, "logp": logp, "lse": lse, "kl": kl, "dlogp": dlogp}
    got = {k: torch.where(w != 0, v, 0.0) for k, v in got.items()}
    got["total"] = (w * got["loss"]).sum()
    return got


def _exact_preference(s, case, step):
    T, R = case["T"], s["logits"].shape[0]
    w, token = s["weight"].double(), s["token"].long()
    lse = torch.cat([(s["logits"][i:i + step].double() / T).logsumexp(1) for i in range(0, R, step)])
    at = s["logits"].gather(1, token[:, None])[:, 0].double() / T
    logp = (at - lse).requires_grad_(True)
    edges = s["seq_start"].tolist()
    terms = w * (logp - s["ref_logp"].double())
    ratio = torch.stack([terms[a:b].sum() for a, b in zip(edges[:-1], edges[1:])])
    z = BETA * (ratio[0::2] - ratio[1::2])
    loss = (torch.nn.functional.softplus(-z, threshold=1000.0) * (1.0 - SMOOTHING)
            + torch.nn.functional.softplus(z, threshold=1000.0) * SMOOTHING)
    dlogp, = torch.autograd.grad(loss.sum(), logp)
    got = {"loss": loss.detach(), "log_ratio": ratio.detach(), "dlogp": dlogp,
           "logp": torch.where(w != 0, logp.detach(), 0.0), "lse": torch.where(w != 0, lse, 0.0)}
    if case["pass"] == "step":
        grad = torch.empty(s["logits"].shape, dtype=torch.float64, device="cuda")
        for i in range(0, R, step):
            b = slice(i, min(R, i + step))
            grad[b] = torch.exp(s["logits"][b].double() / T - lse[b, None]) * (-dlogp[b] / T)[:, None]
        grad.scatter_add_(1, token[:, None], (dlogp / T)[:, None])
        got["grad"] = grad
    return got
