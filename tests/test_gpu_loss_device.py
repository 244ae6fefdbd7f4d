"""The loss calls launch on the current device: logits of another one are refused."""
import pytest
import torch

from test_gpu_losses import B, device_status_stays_clear  # noqa: F401
from test_gpu_loss_workspaces import R, V, calls, x  # noqa: F401

pytestmark = pytest.mark.gpu


def test_logits_of_another_device(B, x, monkeypatch):
    made = calls(B, x)
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_cuda_getDevice", lambda: 1)     # (one GPU here: as if the second were current)
        for name, call in made.items():
            with pytest.raises(ValueError, match="current device"):
                call(None)
    for call in made.values():
        call(None)
