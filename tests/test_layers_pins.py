"""Pins of the float64 oracle of the linear-layer operators (oracle/layers.py):
closed forms, hand-worked values, the format's own table, torch's float64
functions, and every gradient against central differences of its forward
function. CPU only.

Central differences with step h = 1e-4 have an error of about h^2 |f'''| / 6 plus
2^-53 |f| / h: below 1e-7 of the function values here, so 2e-6 is asked for.
"""
import math

import numpy as np
import pytest
import torch

from oracle import layers as L

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def test_activation_values():
    z = np.array([-3.0, -1.0, 0.0, 0.5, 2.0])
    assert np.array_equal(L.act(z, "relu"), [0, 0, 0, 0.5, 2])
    assert L.act(np.array([1.0]), "gelu")[0] == pytest.approx(0.8413447460685429, abs=1e-15)
    assert L.act(np.array([1.0]), "silu")[0] == pytest.approx(1 / (1 + math.exp(-1)), abs=1e-15)
    assert L.act(np.array([1.0]), "gelu_tanh")[0] == pytest.approx(0.841191990608, abs=1e-12)
    t = torch.from_numpy(z)
    f = torch.nn.functional
    for name, ref in (("relu", f.relu(t)), ("gelu", f.gelu(t)), ("silu", f.silu(t)),
                      ("gelu_tanh", f.gelu(t, approximate="tanh"))):
        np.testing.assert_allclose(L.act(z, name), ref.numpy(), rtol=0, atol=1e-15)


@pytest.mark.parametrize("name", ACTS)
def test_activation_slope_is_the_derivative(name):
    z = np.concatenate([np.linspace(-6, 6, 241) + 0.0123, [-0.3, 0.7]])
    h = 1e-4
    fd = (L.act(z + h, name) - L.act(z - h, name)) / (2 * h)
    np.testing.assert_allclose(L.act_slope(z, name), fd, rtol=0, atol=2e-6)


def test_linear_by_hand():
    A = np.array([[1.0, 2.0], [0.0, -1.0]])
    B = np.array([[1.0, 0.0, 2.0], [3.0, 1.0, -1.0]])
    d, z = L.linear(A, B, 2.0, np.array([1.0, 0.0, -1.0]), "relu", np.full((2, 3), 10.0),
                    np.array([1.0, 2.0]), np.array([1.0, 1.0, 0.5]))
    # A B = [[7, 2, 0], [-3, -1, 1]]; times 2, the row and column scales; plus bias
    np.testing.assert_array_equal(z, [[15, 4, -1], [-11, -4, 1]])
    np.testing.assert_array_equal(d, [[25, 14, 10], [10, 10, 11]])


@pytest.mark.parametrize("name", ACTS)
def test_linear_grad_matches_differences(name):
    """d(sum(G * act(A B + bias))) by A, B and bias, from dZ and dbias."""
    r = np.random.default_rng(3)
    A, B, bias, G = (r.standard_normal(s) for s in ((4, 5), (5, 3), (3,), (4, 3)))

    def loss(A, B, bias):
        return (G * L.linear(A, B, 1.0, bias, name)[0]).sum()

    z = L.linear(A, B, 1.0, bias, name)[1]
    dz, db = L.linear_grad(G, z, name)
    h = 1e-4
    for x, grad, put in ((A, dz @ B.T, 0), (B, A.T @ dz, 1), (bias, db, 2)):
        for i in np.ndindex(x.shape):
            p, q = x.copy(), x.copy()
            p[i] += h
            q[i] -= h
            args = [A, B, bias]
            up, down = (loss(*[*args[:put], v, *args[put + 1:]]) for v in (p, q))
            assert grad[i] == pytest.approx((up - down) / (2 * h), abs=2e-6)


def test_rms_norm_closed_forms():
    y, h, s = L.rms_norm(np.array([[3.0, -3.0, 3.0, 3.0]]))
    np.testing.assert_allclose(y, [[1, -1, 1, 1]], atol=1e-15)
    assert s[0] == pytest.approx(1 / 3)
    x = np.random.default_rng(0).standard_normal((5, 33))
    y, _, _ = L.rms_norm(x)
    np.testing.assert_allclose((y * y).mean(1), 1.0, atol=1e-12)
    np.testing.assert_allclose(L.rms_norm(7 * x)[0], y, atol=1e-12)      # scale-free
    np.testing.assert_array_equal(L.rms_norm(x, residual=x)[1], 2 * x)


@pytest.mark.parametrize("gain", [False, True])
def test_rms_norm_grad_matches_differences(gain):
    r = np.random.default_rng(5)
    X, R, G, E = (r.standard_normal((3, 7)) for _ in range(4))
    W = r.standard_normal(7) if gain else None

    def loss(X, W):
        y, h, _ = L.rms_norm(X, W, R, 0.1)
        return (G * y).sum() + (E * h).sum()  # E: the gradient past the norm

    _, H, s = L.rms_norm(X, W, R, 0.1)
    dx, dw = L.rms_norm_grad(G, H, s, W, E)
    h = 1e-4
    for i in np.ndindex(X.shape):
        p, q = X.copy(), X.copy()
        p[i] += h
        q[i] -= h
        assert dx[i] == pytest.approx((loss(p, W) - loss(q, W)) / (2 * h), abs=2e-6)
    if gain:
        for j in range(7):
            p, q = W.copy(), W.copy()
            p[j] += h
            q[j] -= h
            assert dw[j] == pytest.approx((loss(X, p) - loss(X, q)) / (2 * h), abs=2e-6)


def test_e4m3_decoder_is_the_format():
    bits = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(bits.copy()).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    np.testing.assert_array_equal(L.decode_e4m3(bits), ref)
    assert L.decode_e4m3(0x7e) == 448 and L.decode_e4m3(1) == 2.0 ** -9


def test_e4m3_rounding():
    grid = np.unique(L.decode_e4m3(np.arange(127)))
    np.testing.assert_array_equal(L.round_e4m3(grid), grid)
    mid = (grid[1:] + grid[:-1]) / 2
    even = np.where(np.arange(len(mid)) % 2 == 0, grid[:-1], grid[1:])  # ties to even codes
    np.testing.assert_array_equal(L.round_e4m3(mid), even)
    np.testing.assert_array_equal(L.round_e4m3(mid * (1 + 1e-12)), grid[1:])
    np.testing.assert_array_equal(L.round_e4m3(mid * (1 - 1e-12)), grid[:-1])
    assert L.round_e4m3(1e9) == 448 and L.round_e4m3(-1e9) == -448
    x = np.random.default_rng(1).standard_normal(4000).astype(np.float32) * 30
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    np.testing.assert_array_equal(L.round_e4m3(x), ref)


def test_quantise_uses_the_whole_range():
    y = np.random.default_rng(2).standard_normal((6, 50))
    y[3] = 0
    q, s = L.quantise_e4m3(y)
    assert s[3] == 0 and not q[3].any()
    live = [0, 1, 2, 4, 5]
    np.testing.assert_array_equal(np.abs(q[live]).max(1), 448)
    assert (np.abs(q * s[:, None] - y) <= 2.0 ** -4 * np.abs(y) + s[:, None] * 2.0 ** -10).all()
