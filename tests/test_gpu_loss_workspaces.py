"""The binding's checks of a caller's workspace: its memory is what the kernels write."""
import numpy as np
import pytest
import torch

from test_gpu_losses import B, device_status_stays_clear, f32, i32, logits  # noqa: F401

pytestmark = pytest.mark.gpu

R, V = 3, 20004


def calls(B, x):
    tok, one = i32([1, 2, 3]), f32([1, 1, 1])
    idx, t = i32([[0, 1], [2, 3], [4, 5]]), f32(np.zeros((3, 2)))
    lse = torch.logsumexp(x.float(), 1)
    return {
        "topk": lambda ws: B.dg_row_topk(x, 5, ws=ws)["values"],
        "logp": lambda ws: B.dg_token_logp(x, tok, ws=ws)["logp"],
        "logp backward": lambda ws: B.dg_token_logp_backward(x, tok, lse, one, ws=ws),
        "distill": lambda ws: B.dg_distill_loss(x, idx, t, grad=True, ws=ws)["grad"],
        "distill backward": lambda ws: B.dg_distill_loss_backward(x, idx, t, lse, ws=ws),
        "policy": lambda ws: B.dg_policy_loss(x, tok, -one, one, grad=True, ws=ws)["grad"],
        "preference": lambda ws: B.dg_preference_loss(x, tok, None, i32([0, 1, 3]), grad=True, ws=ws)["grad"],
    }


@pytest.fixture
def x(B):
    return logits(np.random.default_rng(0), R, V, "f32")[0]


def test_workspaces_that_are_not_their_size(B, x):
    """On the host, a broadcast, and every other byte."""
    n = max(B.dg_row_loss_workspace_size(R, V), B.dg_row_topk_workspace_size(R, V, 5))
    bad = [torch.empty(n, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(n),
           torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]]
    for name, call in calls(B, x).items():
        for ws in bad:
            with pytest.raises(ValueError, match="workspace"):
                call(ws)


def test_a_workspace_of_any_type_counts_in_bytes(B, x):
    n = max(B.dg_row_loss_workspace_size(R, V), B.dg_row_topk_workspace_size(R, V, 5))
    ws = torch.empty((n + 7) // 8, dtype=torch.float64, device="cuda")
    for name, call in calls(B, x).items():
        assert torch.equal(call(ws), call(None)), name
        with pytest.raises(B.DgError, match="below"):
            call(ws[:1])


def test_rows_of_one_tile_ignore_it(B):
    x = logits(np.random.default_rng(0), R, 100, "f32")[0]
    for name, call in calls(B, x).items():
        if name not in ("topk", "distill backward"):
            assert torch.equal(call(torch.empty(0)), call(None)), name
