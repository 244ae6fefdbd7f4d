"""dg_row_topk's refusal of more logits than its counters hold, on the host (no GPU)."""
import ctypes

import pytest

P = ctypes.c_void_p(256)


@pytest.fixture(scope="module")
def lib():
    from denoising_sampler_step_gb300 import build
    build.build()
    from denoising_sampler_step_gb300 import binding
    return binding.lib


@pytest.mark.parametrize("R,V,dtype", [(1 << 28, 1 << 27, 0), (1 << 28, 16385, 0), (1 << 20, 1 << 23, 0), (1 << 28, 32769, 1)])
def test_more_rows_than_can_be_counted(lib, R, V, dtype):
    ld = (V + 7) // 8 * 8
    assert lib.dg_row_topk(P, dtype, R, V, ld, 5, 1.0, P, P, 5, P, P, 1 << 50, None) == 2
    assert b"16 TiB" in lib.dg_last_error()
    assert lib.dg_row_topk_workspace_size(R, V, 5, dtype) == 0
    assert lib.dg_row_topk_workspace_size(1 << 61, 100, 5, dtype) == 0
