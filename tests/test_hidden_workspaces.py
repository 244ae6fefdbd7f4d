"""The hidden stream's workspaces: one for the largest call serves every smaller one (on the host, no GPU)."""
import pytest


@pytest.fixture(scope="module")
def L():
    from denoising_sampler_step_gb300 import build
    build.build()
    from denoising_sampler_step_gb300 import binding
    return binding.lib


# around the sizes where the embedding gradient's plan changes: R ceil(d / 256) = 65,536
R = sorted({1, 15, 16, 17, 18, 31, 32, 33, 256, 257, 1000, 3855, 3856, 4096, 5000, 5461, 5462, 5957, 5958, 8192, 16383, 16384,
            20001, 32767, 32768, 40000, 65535, 65536, 65537, 100000, 1 << 20})
D = sorted({1, 7, 8, 255, 256, 257, 512, 513, 1001, 1024, 1025, 2048, 2049, 2816, 4096, 8200, 65536, 900000, 986880, 986881,
            1 << 20})


def test_the_embedding_gradients(L):
    size = {(r, d): L.dg_token_embed_backward_workspace_size(r, 1000, d) for r in R for d in D}
    for r0, r1 in zip(R, R[1:]):
        assert all(0 < size[r0, d] <= size[r1, d] for d in D), (r0, r1)
    for d0, d1 in zip(D, D[1:]):
        assert all(0 < size[r, d0] <= size[r, d1] for r in R), (d0, d1)
    # a slice's length does not count
    assert L.dg_token_embed_backward_workspace_size(8192, 0, 2816) == size[8192, 2816]


def test_the_norm_gradients(L):
    widths = [d for d in D if d <= 32768]
    size = {(r, d): L.dg_rms_norm_backward_workspace_size(r, d) for r in R for d in widths}
    for r0, r1 in zip(R, R[1:]):
        assert all(0 < size[r0, d] <= size[r1, d] for d in widths), (r0, r1)
    for d0, d1 in zip(widths, widths[1:]):
        assert all(0 < size[r, d0] <= size[r, d1] for r in R), (d0, d1)
