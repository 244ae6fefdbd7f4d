"""A small training run over the sampler: `python -m denoising_sampler_step_gb300.finetune`.

The "model" is one hidden vector per canvas position times a fixed embedding table, so that its
logits are what the sampler's calls take; what is trained is the hidden vectors.  Three stages, as
a diffusion model's sampler is tuned in earnest:

1. distillation: a teacher's logits are reduced to their top entries (dg_row_topk), and the student
   is brought to them (dg_distill_loss, losses and gradient from one read of the logits);
2. policy: candidates are drawn from the student with the sampler's own draw (dg_row_sample), whose
   log-probabilities are the behaviour policy's, and rewarded (training.policy_loss);
3. preference: canvases of rewarded and of unrewarded tokens form pairs (training.preference_loss).
"""
from __future__ import annotations

import argparse

import torch

from . import binding as B
from . import inputs, training


def run(steps: int = 60, K: int = 64, seed: int = 0, log=print) -> dict:
    """Runs the three stages and returns what each measured before and after."""
    wl = inputs.WORKLOADS["tiny"]
    R, V, d = wl.R, wl.V, wl.d
    g = torch.Generator(device="cuda").manual_seed(seed)
    # entries of about unit size: logits of a few nats from hidden vectors of unit size
    table = torch.randn(V, d, generator=g, device="cuda") / d ** 0.5
    hidden = torch.zeros(R, d, device="cuda", requires_grad=True)
    report = {}

    # 1. distillation from the top entries of a teacher
    teacher_hidden = 3.0 * torch.randn(R, d, generator=g, device="cuda")
    top = B.dg_row_topk(teacher_hidden @ table.T, K, lse=True)
    weight = torch.full((R,), 1.0 / R, device="cuda")
    opt = torch.optim.Adam([hidden], lr=0.1)
    out = {}
    for step in range(steps):
        opt.zero_grad()
        logits = hidden @ table.T
        B.dg_distill_loss(logits.detach(), top["indices"], top["values"], top["lse"], weight=weight, grad=True, out=out)
        logits.backward(out["grad"])
        opt.step()
        if step == 0:
            first = out["loss"].mean()
    report["distill"] = (float(first), float(out["loss"].mean()))

    # 2. a policy rewarded for tokens of the vocabulary's first half, held near where it started
    reward_of = (torch.arange(V, device="cuda") < V // 2).float()
    reference = hidden.detach().clone()
    opt = torch.optim.Adam([hidden], lr=0.02)
    rewards = []
    for step in range(steps):
        with torch.no_grad():
            logits = hidden @ table.T
            draw = B.dg_row_sample(logits, 1.0, seed=seed, offset=step)
            ref = B.dg_token_logp(reference @ table.T, draw["candidate"])["logp"]
            reward = reward_of[draw["candidate"].long()]
            rewards.append(reward.mean())
        for _ in range(2):  # two updates on one draw: the second one's ratios are clipped
            opt.zero_grad()
            loss, _ = training.policy_loss(hidden @ table.T, draw["candidate"], draw["log_p"], reward - reward.mean(),
                                           ref_logp=ref, kl_coef=0.01)
            loss.mean().backward()
            opt.step()
    p = torch.softmax(hidden.detach() @ table.T, 1) @ reward_of
    p0 = torch.softmax(reference @ table.T, 1) @ reward_of
    report["policy"] = (float(p0.mean()), float(p.mean()))

    # 3. pairs: each position's hidden vector stands for two answers of one canvas
    tokens = torch.randint(V // 2, (2, R), generator=g, device="cuda")
    tokens[1] += V // 2                      # preferred: the first half again
    token = tokens.reshape(-1).to(torch.int32)
    start = torch.tensor([0, R, 2 * R], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        ref = B.dg_token_logp((hidden @ table.T).repeat(2, 1), token)["logp"]
    margins = []
    for step in range(steps):
        opt.zero_grad()
        logits = (hidden @ table.T).repeat(2, 1)
        loss, ratio = training.preference_loss(logits, token, ref, start)
        loss.sum().backward()
        opt.step()
        margins.append(ratio[0] - ratio[1])
    report["preference"] = (float(margins[0]), float(margins[-1]))

    B.dg_get_device_status()
    log(f"distillation   loss per position   {report['distill'][0]:.4f} -> {report['distill'][1]:.4f} nats")
    log(f"policy         rewarded mass       {report['policy'][0]:.4f} -> {report['policy'][1]:.4f}")
    log(f"preference     log ratio margin    {report['preference'][0]:.4f} -> {report['preference'][1]:.4f}")
    return report


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--top", type=int, default=64, help="teacher entries kept per position")
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    run(a.steps, a.top, a.seed)


if __name__ == "__main__":
    main()
