"""What the loss calls say about rows off a 16-byte boundary, on the host (no GPU)."""
import ctypes

import pytest

P, Q, BIG = ctypes.c_void_p(256), ctypes.c_void_p(264), ctypes.c_void_p(1 << 40)
WS = [P, 1 << 30, None]


@pytest.fixture(scope="module")
def lib():
    from denoising_sampler_step_gb300 import build
    build.build()
    from denoising_sampler_step_gb300 import binding
    return binding.lib


@pytest.mark.parametrize("dtype,per", [(0, b"4"), (1, b"8")])
def test_the_message_says_what_to_do(lib, dtype, per):
    for ptr, ld in ((P, 50257), (Q, 50264)):
        assert lib.dg_token_logp(ptr, dtype, 4, 50257, ld, P, 1.0, None, P, P, *WS) == 2
        assert b"multiple of " + per + b" elements" in lib.dg_last_error()
    assert lib.dg_token_logp_backward(P, dtype, 4, 50257, 50264, P, 1.0, P, P, None, BIG, 50258, *WS) == 2
    assert b"grad rows" in lib.dg_last_error() and b"multiple of " + per + b" elements" in lib.dg_last_error()
