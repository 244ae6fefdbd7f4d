"""Numbers of the differentiable functions given as tensors that require a gradient are refused: it would be lost."""
import pytest
import torch

from test_training_refusals import T, tensors  # noqa: F401

NUMBERS = [("token_logp", "temperature"), ("distill_loss", "temperature"), ("policy_loss", "clip_low"),
           ("policy_loss", "clip_high"), ("policy_loss", "kl_coef"), ("policy_loss", "temperature"),
           ("preference_loss", "beta"), ("preference_loss", "label_smoothing"), ("preference_loss", "temperature"),
           ("token_embed", "gamma"), ("rms_norm", "eps"), ("rms_norm", "weight_offset")]


def call(T, name, device, **number):
    x, tok, v, idx, t, start = tensors(device)
    args = {"token_logp": (x, tok), "distill_loss": (x, idx, t), "policy_loss": (x, tok, v, -v),
            "preference_loss": (x, tok, v, start), "token_embed": (x, tok % 4), "rms_norm": (x, None, x)}[name]
    o = getattr(T, name)(*args, **number)
    return o[0] if isinstance(o, tuple) else o


@pytest.mark.parametrize("name,number", NUMBERS)
def test_a_number_that_requires_a_gradient(T, name, number):
    with pytest.raises(ValueError, match=f"{number} requires a gradient"):
        call(T, name, "cpu", **{number: torch.tensor(0.25, requires_grad=True)})


@pytest.mark.gpu
@pytest.mark.parametrize("name,number", NUMBERS)
def test_a_number_as_a_tensor(T, name, number):
    """Without a gradient asked for it is the number that it holds."""
    want = call(T, name, "cuda", **{number: 0.25})
    assert torch.equal(call(T, name, "cuda", **{number: torch.tensor(0.25)}), want)
    with torch.no_grad():
        assert torch.equal(call(T, name, "cuda", **{number: torch.tensor(0.25, requires_grad=True).detach()}), want)
