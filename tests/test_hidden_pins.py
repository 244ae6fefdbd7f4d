"""The hidden stream's oracle against what does not share its formulas: differences, one-hot products, torch."""
import numpy as np
import pytest
import torch

from oracle import e4m3_decode, hidden_oracle as H


def test_the_lookup_is_a_one_hot_product():
    rng = np.random.default_rng(0)
    W, tok = rng.normal(size=(7, 5)), np.array([0, 6, 3, 3, -1, 2])
    hot = np.zeros((6, 7))
    hot[tok >= 0, tok[tok >= 0]] = 1
    assert np.allclose(H.token_embed(W, tok, 2.5), 2.5 * hot @ W, atol=1e-15)
    # slices of the vocabulary add up to it
    parts = [H.token_embed(W[a:b], tok, 2.5, a, b) for a, b in ((0, 2), (2, 2), (2, 7))]
    assert np.array_equal(sum(parts), H.token_embed(W, tok, 2.5))
    g = rng.normal(size=(6, 5))
    o = H.token_embed_backward(g, tok, 2.5, 0, 7)
    assert np.allclose(o["grad"], 2.5 * hot.T @ g, atol=1e-14) and o["count"].tolist() == [1, 0, 1, 2, 0, 0, 1]


@pytest.mark.parametrize("R,d", [(1, 1), (3, 7), (5, 16)])
def test_the_norms_gradient_against_differences(R, d):
    rng = np.random.default_rng(d)
    x, res, w, g, up = (rng.normal(size=s) for s in ((R, d), (R, d), d, (R, d), (R, d)))

    def loss(x, w):
        o = H.rms_norm(x, res, w, 1e-3)
        return np.sum(g * o["out"]) + np.sum(up * o["hidden"])
    o = H.rms_norm(x, res, w, 1e-3)
    b = H.rms_norm_backward(g, o["hidden"], o["rstd"], w, up)
    t = 1e-6
    for i in range(R):
        for j in range(d):
            e = np.zeros((R, d))
            e[i, j] = t
            assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * t) - b["grad"][i, j]) < 1e-7 * (1 + abs(b["grad"][i, j]))
    for j in range(d):
        e = np.zeros(d)
        e[j] = t
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * t) - b["grad_weight"][j]) < 1e-6


def test_the_norm_against_torch():
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(4, 33, generator=g, dtype=torch.float64), torch.randn(33, generator=g, dtype=torch.float64)
    ref = torch.nn.functional.rms_norm(x, (33,), w, 1e-5)
    assert np.allclose(H.rms_norm(x.numpy(), None, w.numpy(), 1e-5)["out"], ref.numpy(), atol=1e-13)


def test_codes_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(e4m3_decode(codes), ref, equal_nan=True)
