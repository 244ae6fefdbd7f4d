"""The norm's 8-bit codes: the ones that its own y and scale have by the definition, e4m3(y / scale) with the quotient
rounded once, bit for bit.  No tolerance: y is the same call's in fp32, scale = max|y| / 448 and the quotient are IEEE
divisions, taken on the CPU here.  Operands of 8 bits make many quotients ties between two codes."""
import numpy as np
import pytest
import torch

from test_gpu_hidden import B, device_status_stays_clear, place  # noqa: F401

pytestmark = pytest.mark.gpu


def check(B, x, residual, w, offset):
    c = B.dg_rms_norm(x, w, residual=residual, weight_offset=offset, dtype=torch.uint8)
    o = B.dg_rms_norm(x, w, residual=residual, weight_offset=offset, dtype=torch.float32)
    assert torch.equal(c["rstd"], o["rstd"])
    y = o["out"].cpu().numpy()
    scale = np.abs(y).max(1) / np.float32(448)
    assert np.array_equal(c["scale"].cpu().numpy(), scale)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where(scale[:, None] > 0, y / scale[:, None], np.float32(0))
    q = q.clip(-448, 448)   # (a scale of few bits, near the smallest number, may be up to a third too small)
    want = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8)
    bad = (c["out"].cpu() != want).any(1)
    assert not bad.any(), f"codes differ in {int(bad.sum())} of {len(bad)} rows"
    return scale


@pytest.mark.parametrize("R,d", [(1, 2816), (3001, 264), (6001, 2816), (40, 8200), (700, 999)])
@pytest.mark.parametrize("layout", ["wide", "odd"])
@pytest.mark.parametrize("res", ["bf16", "f32", None])
def test_codes_are_the_quotients(B, R, d, layout, res):
    g = torch.Generator().manual_seed(R + d)
    size = torch.exp(torch.randn(R, 1, generator=g))
    x, _ = place(size * torch.randn(R, d, generator=g), "bf16", layout)
    r, _ = place(size * torch.randn(R, d, generator=g), res, layout) if res else (None, None)
    check(B, x, r, (0.3 * torch.randn(d, generator=g)).bfloat16().cuda(), 1.0)


@pytest.mark.parametrize("layout", ["wide", "odd"])
def test_codes_of_rows_whose_scale_is_near_the_ends(B, layout):
    """Scales down to the smallest numbers and up to the largest, on either side of every choice between a
    product and a division."""
    g = torch.Generator().manual_seed(7)
    x, _ = place(torch.randn(30, 520, generator=g), "f32", layout)
    seen = []
    for e in (-149, -140, -130, -127, -126, -125, -100, -82, -81, -80, -79, -78, -60, 0, 60, 100, 120, 125):
        w = torch.ldexp(1 + torch.rand(520, generator=g), torch.tensor(e)).cuda()
        seen.append(check(B, x, None, w, 0.0))
    seen = np.concatenate(seen)
    assert seen.min() < 2.0 ** -140 and seen.max() > 2.0 ** 115
