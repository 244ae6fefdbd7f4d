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
