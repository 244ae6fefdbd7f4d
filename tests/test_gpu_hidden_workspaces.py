"""One workspace for call after call: nothing of one call's inputs or parts is seen by the next."""
import pytest
import torch

from test_gpu_hidden import B, device_status_stays_clear  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,d", [(3001, 1153), (6001, 1160), (40, 8200), (700, 264)])
def test_the_norms_gradient_again_and_again(B, R, d):
    """Weight gradients of inputs that alternate, without a pause between the calls, each that of a call by itself."""
    g = torch.Generator(device="cuda").manual_seed(R)
    per = (d + 7) // 8 * 8
    h, w = torch.randn(R, per, generator=g, device="cuda")[:, :d], torch.randn(d, generator=g, device="cuda")
    rstd = (h.square().mean(1) + 1e-6).rsqrt()
    grads = [torch.randn(R, per, generator=g, device="cuda")[:, :d] for _ in range(3)]
    ref = []
    for t in grads:
        ref.append(B.dg_rms_norm_backward(t, h, rstd, w)["grad_weight"])
        torch.cuda.synchronize()
    ws = B.norm_workspace(R, d, "cuda")
    out = torch.empty(R, per, device="cuda")[:, :d]
    got = torch.empty(30, 3, d, device="cuda")
    for i in range(30):
        for k, t in enumerate(grads):
            B.dg_rms_norm_backward(t, h, rstd, w, ws=ws, out={"grad": out, "grad_weight": got[i, k]})
    for k in range(3):
        assert (got[:, k] == ref[k]).all()


@pytest.mark.parametrize("most,calls", [((8192, 2816), [(5000, 2816), (5957, 2816), (8192, 2500), (6553, 2560), (17, 2816), (1, 1)]),
                                        ((40000, 1001), [(40000, 256), (40000, 257), (16383, 1001), (32767, 512), (300, 40)])])
def test_a_workspace_for_the_largest_call_serves_smaller_ones(B, most, calls):
    g = torch.Generator(device="cuda").manual_seed(1)
    need = B.dg_token_embed_backward_workspace_size(most[0], 500, most[1])
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    for R, d in calls:
        grad = torch.randn(R, (d + 7) // 8 * 8, generator=g, device="cuda")[:, :d]
        tok = torch.randint(500, (R,), generator=g, device="cuda").int()
        tok[torch.rand(R, generator=g, device="cuda") < 0.5] = 77
        got = B.dg_token_embed_backward(grad, tok, 500, ws=ws[:need])
        assert torch.equal(got, B.dg_token_embed_backward(grad, tok, 500))
        assert (ws[need:] == 0xFF).all()
        # (n + 3) roundings of 2^-24 of the terms' magnitudes
        want = torch.zeros(500, d, dtype=torch.float64, device="cuda").index_add_(0, tok, grad.double())
        size = torch.zeros(500, d, dtype=torch.float64, device="cuda").index_add_(0, tok, grad.double().abs())
        n = torch.bincount(tok, minlength=500)[:, None]
        assert ((got - want).abs() <= (n + 3) * 2.0 ** -24 * size).all()
