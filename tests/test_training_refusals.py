"""What the differentiable losses refuse instead of dropping a gradient in silence."""
import pytest
import torch


@pytest.fixture(scope="module")
def T():
    from denoising_sampler_step_gb300 import build
    build.build()
    from denoising_sampler_step_gb300 import training
    return training


def tensors(device):
    x = torch.linspace(-2, 2, 4 * 24, device=device).view(4, 24)
    tok = torch.tensor([1, 5, 9, 23], dtype=torch.int32, device=device)
    v = torch.full((4,), -2.0, device=device)
    idx = torch.arange(8, dtype=torch.int32, device=device).view(4, 2)
    start = torch.tensor([0, 2, 4], dtype=torch.int32, device=device)
    return x, tok, v, idx, torch.zeros(4, 2, device=device), start


def calls(T, x, tok, v, idx, t, start):
    return {
        "token": lambda **k: T.token_logp(x, tok),
        "distill": lambda teacher=t, teacher_lse=-v: T.distill_loss(x, idx, teacher, teacher_lse),
        "policy": lambda old_logp=v, advantage=-v, ref_logp=v: T.policy_loss(x, tok, old_logp, advantage, ref_logp,
                                                                            kl_coef=0.1)[0],
        "preference": lambda ref_logp=v, weight=-v: T.preference_loss(x, tok, ref_logp, start, weight=weight)[0],
    }


ARGUMENTS = [("distill", "teacher"), ("distill", "teacher_lse"), ("policy", "old_logp"), ("policy", "advantage"),
             ("policy", "ref_logp"), ("preference", "ref_logp"), ("preference", "weight")]


@pytest.mark.parametrize("call,name", ARGUMENTS)
def test_arguments_that_require_a_gradient(T, call, name):
    x, tok, v, idx, t, start = tensors("cpu")
    arg = (t if name == "teacher" else v).clone().requires_grad_(True)
    with pytest.raises(ValueError, match=f"{name} requires a gradient"):
        calls(T, x, tok, v, idx, t, start)[call](**{name: arg})


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["token", "distill", "policy", "preference"])
def test_second_derivatives(T, call):
    x, *rest = tensors("cuda")
    x.requires_grad_(True)
    f = calls(T, x, *rest)[call]
    first, = torch.autograd.grad(f().sum(), x)
    assert first.abs().sum() > 0 and not first.requires_grad
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad(f().sum(), x, create_graph=True)


@pytest.mark.gpu
@pytest.mark.parametrize("call,name", ARGUMENTS)
def test_no_gradient_is_asked_for(T, call, name):
    """Under no_grad such an argument is a plain tensor."""
    x, tok, v, idx, t, start = tensors("cuda")
    arg = (t if name == "teacher" else v).clone()
    want = calls(T, x, tok, v, idx, t, start)[call](**{name: arg})
    with torch.no_grad():
        got = calls(T, x, tok, v, idx, t, start)[call](**{name: arg.requires_grad_(True)})
    assert torch.equal(got, want)
