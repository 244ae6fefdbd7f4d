"""Distillation with long lists of a teacher's entries, against the float64 oracle; tolerances as derived in
test_gpu_losses.py.

A stage of the ring holds a tile and its list: beside the longest lists only two stages of a row of 64 KB fit.
Over longer rows, lists above 256 entries have tiles of their own size.
"""
import numpy as np
import pytest

from test_gpu_losses import B, check_distill, device_status_stays_clear, distill_case, mask_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,dtype", [(15940, "f32"), (16384, "f32"), (16387, "f32"), (31880, "bf16"), (32000, "bf16"),
                                     (32003, "bf16"), (32768, "bf16"), (32775, "bf16")])
@pytest.mark.parametrize("K", [881, 882, 900, 1024])
@pytest.mark.parametrize("tail", [False, True])
def test_rows_of_one_tile(B, V, dtype, K, tail):
    """Losses and gradient in one pass, without a workspace."""
    assert not B.dg_row_loss_needs_workspace(V, {"f32": B.DG_F32, "bf16": B.DG_BF16}[dtype])
    rng, x, xf, idx, t, lse = distill_case(5, V, K, dtype, 1.2, tail)
    idx[1, 3::2] = -1
    w = mask_of(rng, 5)
    w[:2] = 1.0, 0.5
    check_distill(B, x, xf, idx, t, lse, 1.2, w, dtype)


@pytest.mark.parametrize("dtype,V", [("f32", 16384), ("bf16", 32768)])
def test_more_rows_of_one_tile_than_stages(B, dtype, V):
    """Several rows for every CTA, through the two stages in turn."""
    rng, x, xf, idx, t, lse = distill_case(500, V, 1024, dtype, 1.0, True, pad=1)
    check_distill(B, x, xf, idx, t, lse, 1.0, mask_of(rng, 500), dtype, backward=False)


@pytest.mark.parametrize("V", [100003, 262144])
@pytest.mark.parametrize("K", [255, 257, 300, 512, 1024])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tail", [False, True])
def test_split_rows(B, V, K, dtype, tail):
    rng, x, xf, idx, t, lse = distill_case(7, V, K, dtype, 1.2, tail)
    idx[1] = np.arange(V // 2, V // 2 + K)     # a list that one or two tiles hold whole
    idx[2, ::3] = -1
    w = mask_of(rng, 7)
    w[:3] = 1.0, 0.5, 2.0
    check_distill(B, x, xf, idx, t, lse, 1.2, w, dtype)
