"""The losses on the sampler's logits as differentiable functions.

Each function returns one loss per row (or pair) and can stand in any autograd expression of the
logits: the forward pass is one call of the library (losses and the log-sum-exp), the backward
pass another that turns the saved log-sum-exp and the upstream gradients into the logits'
gradient.  A training loop that knows its row weights beforehand gets both from one read of the
logits with the binding's own calls (`grad=True`, weights in `weight`).

`mask` [R] (bool or any type: nonzero counts) leaves rows out: their logits are not read, their
loss is 0 and their gradient 0.

The functions differentiate once and in the logits alone.  Another argument that requires a gradient
is an error (detach it), and so is `create_graph=True`: what would be lost is not lost in silence.
"""
from __future__ import annotations

import torch

from . import binding as B


def _weight(mask: torch.Tensor | None) -> torch.Tensor | None:
    return None if mask is None else (mask != 0).float()


def _upstream(g: torch.Tensor, weight: torch.Tensor | None) -> torch.Tensor:
    """Upstream gradients of the rows that count, contiguous."""
    g = g if weight is None else torch.where(weight != 0, g, 0.0)
    return g.float().contiguous()


def _constants(**tensors) -> None:
    """Refuses arguments whose gradient would be dropped."""
    for name, t in tensors.items():
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} requires a gradient, and the loss is differentiable in the logits alone: "
                             f"pass {name}.detach()")


def _first_order() -> None:
    """Refuses a backward pass that is to be differentiated (autograd records it only then)."""
    if torch.is_grad_enabled():
        raise RuntimeError("the losses on logits have first derivatives only: with create_graph=True their "
                           "gradient would count as a constant")


class _TokenLogp(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, token, temperature, weight):
        o = B.dg_token_logp(logits, token, temperature=temperature, weight=weight)
        ctx.save_for_backward(logits, token, o["lse"], weight)
        ctx.temperature = temperature
        return o["logp"]

    @staticmethod
    def backward(ctx, g):
        _first_order()
        logits, token, lse, weight = ctx.saved_tensors
        grad = B.dg_token_logp_backward(logits, token, lse, _upstream(g, weight), temperature=ctx.temperature)
        return grad, None, None, None


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, indices, teacher, teacher_lse, temperature, weight):
        o = B.dg_distill_loss(logits, indices, teacher, teacher_lse=teacher_lse, temperature=temperature,
                              weight=weight)
        ctx.save_for_backward(logits, indices, teacher, teacher_lse, o["lse"], o.get("tail_logp"), weight)
        ctx.temperature = temperature
        return o["loss"]

    @staticmethod
    def backward(ctx, g):
        _first_order()
        logits, indices, teacher, teacher_lse, lse, tail_logp, weight = ctx.saved_tensors
        grad = B.dg_distill_loss_backward(logits, indices, teacher, lse, _upstream(g, weight),
                                          teacher_lse=teacher_lse, tail_logp=tail_logp,
                                          temperature=ctx.temperature)
        return grad, None, None, None, None, None


class _Policy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, token, old_logp, advantage, ref_logp, clip_low, clip_high, kl_coef, temperature,
                weight):
        o = B.dg_policy_loss(logits, token, old_logp, advantage, ref_logp=ref_logp, clip_low=clip_low,
                             clip_high=clip_high, kl_coef=kl_coef, temperature=temperature, weight=weight)
        ctx.save_for_backward(logits, token, o["lse"], o["dlogp"], weight)
        ctx.temperature = temperature
        ctx.mark_non_differentiable(o["logp"], o["kl"], o["clipped"])
        return o["loss"], o["logp"], o["kl"], o["clipped"]

    @staticmethod
    def backward(ctx, g, *_):
        _first_order()
        logits, token, lse, dlogp, weight = ctx.saved_tensors
        grad = B.dg_token_logp_backward(logits, token, lse, dlogp, scale=_upstream(g, weight),
                                        temperature=ctx.temperature)
        return (grad,) + (None,) * 9


class _Preference(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, token, ref_logp, seq_start, beta, label_smoothing, temperature, weight):
        o = B.dg_preference_loss(logits, token, ref_logp, seq_start, beta=beta, label_smoothing=label_smoothing,
                                 temperature=temperature, weight=weight)
        ctx.save_for_backward(logits, token, seq_start, o["lse"], o["dlogp"])
        ctx.temperature = temperature
        ctx.mark_non_differentiable(o["log_ratio"])
        return o["loss"], o["log_ratio"]

    @staticmethod
    def backward(ctx, g, _):
        _first_order()
        logits, token, seq_start, lse, dlogp = ctx.saved_tensors
        # the pair each row belongs to (rows in no pair have dlogp 0, whatever their scale)
        rows = torch.arange(logits.shape[0], dtype=torch.int32, device=logits.device)
        pair = (torch.searchsorted(seq_start, rows, right=True) - 1).div(2, rounding_mode="floor")
        scale = g.float()[pair.clamp(0, max(0, g.shape[0] - 1))].contiguous() if g.shape[0] else None
        grad = B.dg_token_logp_backward(logits, token, lse, dlogp, scale=scale, temperature=ctx.temperature)
        return (grad,) + (None,) * 7


def token_logp(logits: torch.Tensor, token: torch.Tensor, temperature: float = 1.0,
               mask: torch.Tensor | None = None) -> torch.Tensor:
    """ln softmax(logits / T)[token] per row [R], differentiable in the logits."""
    return _TokenLogp.apply(logits, token, temperature, _weight(mask))


def distill_loss(logits: torch.Tensor, indices: torch.Tensor, teacher: torch.Tensor,
                 teacher_lse: torch.Tensor | None = None, temperature: float = 1.0,
                 mask: torch.Tensor | None = None) -> torch.Tensor:
    """Distillation loss per row [R] from a teacher's top logits (binding.dg_distill_loss)."""
    _constants(teacher=teacher, teacher_lse=teacher_lse)
    return _Distill.apply(logits, indices, teacher, teacher_lse, temperature, _weight(mask))


def policy_loss(logits: torch.Tensor, token: torch.Tensor, old_logp: torch.Tensor, advantage: torch.Tensor,
                ref_logp: torch.Tensor | None = None, clip_low: float = 0.2, clip_high: float = 0.2,
                kl_coef: float = 0.0, temperature: float = 1.0,
                mask: torch.Tensor | None = None) -> tuple[torch.Tensor, dict]:
    """(loss per row [R], {logp, kl, clipped}) of the clipped policy loss (binding.dg_policy_loss)."""
    _constants(old_logp=old_logp, advantage=advantage, ref_logp=ref_logp)
    loss, logp, kl, clipped = _Policy.apply(logits, token, old_logp, advantage, ref_logp, clip_low, clip_high,
                                            kl_coef, temperature, _weight(mask))
    return loss, {"logp": logp, "kl": kl, "clipped": clipped}


def preference_loss(logits: torch.Tensor, token: torch.Tensor, ref_logp: torch.Tensor | None,
                    seq_start: torch.Tensor, beta: float = 0.1, label_smoothing: float = 0.0,
                    temperature: float = 1.0, weight: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(loss per pair [P], log ratios per sequence [2P]) of the preference loss
    (binding.dg_preference_loss); `weight` [R] masks tokens or normalises by length."""
    _constants(ref_logp=ref_logp, weight=weight)
    return _Preference.apply(logits, token, ref_logp, seq_start, beta, label_smoothing, temperature, weight)
