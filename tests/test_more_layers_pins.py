"""The float64 definitions of the gated layer, the block-scaled products and the
layer norm (oracle/layers.py), pinned by closed forms and central differences."""
import numpy as np
import pytest

from oracle import layers as L


def differences(loss, args, grads, h=1e-4, atol=2e-6):
    """grads[i] is the gradient of loss(*args) at args[i]."""
    for put, grad in enumerate(grads):
        for i in np.ndindex(args[put].shape):
            up, down = ([a.copy() for a in args] for _ in range(2))
            up[put][i] += h
            down[put][i] -= h
            assert grad[i] == pytest.approx((loss(*up) - loss(*down)) / (2 * h), abs=atol)


def test_layer_norm_closed_forms():
    y, h, m, s = L.layer_norm(np.array([[1.0, 3.0, 1.0, 3.0]]))
    np.testing.assert_allclose(y, [[-1, 1, -1, 1]], atol=1e-15)
    assert m[0] == 2 and s[0] == pytest.approx(1)
    x = np.random.default_rng(0).standard_normal((5, 33))
    y, h, _, _ = L.layer_norm(x, residual=x)
    np.testing.assert_array_equal(h, 2 * x)
    np.testing.assert_allclose(y.mean(1), 0, atol=1e-14)
    np.testing.assert_allclose((y * y).mean(1), 1, atol=1e-12)
    np.testing.assert_allclose(L.layer_norm(7 * x + 3)[0], y, atol=1e-12)  # scale and shift
    w, b = np.arange(33.0), np.linspace(-1, 1, 33)
    np.testing.assert_allclose(L.layer_norm(x, w, b)[0], y * w + b, atol=1e-12)


@pytest.mark.parametrize("gain", [False, True])
def test_layer_norm_grad_matches_differences(gain):
    r = np.random.default_rng(5)
    X, R, G, E = (r.standard_normal((3, 7)) for _ in range(4))
    W, b = (r.standard_normal(7) for _ in range(2))

    def loss(X, b, W=W):
        y, h, _, _ = L.layer_norm(X, W if gain else None, b, R, 0.1)
        return (G * y).sum() + (E * h).sum()  # E: the gradient past the norm

    _, H, m, s = L.layer_norm(X, W if gain else None, b, R, 0.1)
    dx, dw, db = L.layer_norm_grad(G, H, m, s, W if gain else None, E)
    differences(loss, [X, b, W], [dx, db, dw] if gain else [dx, db])


def test_gated_closed_forms():
    r = np.random.default_rng(1)
    A, B = r.standard_normal((3, 4)), r.standard_normal((4, 5))
    D, G, U = L.gated(A, B, 2 * B, act_name="none")
    np.testing.assert_allclose(D, 2 * (A @ B) ** 2)
    np.testing.assert_allclose(G, A @ B)
    one = L.gated(A, B, 0 * B, 0.5, None, np.ones(5), "silu")[0]  # U = 1: the activation alone
    np.testing.assert_allclose(one, L.linear(A, B, 0.5, act_name="silu")[0])


@pytest.mark.parametrize("name", ["none", "gelu", "gelu_tanh", "silu"])
def test_gated_grad_matches_differences(name):
    r = np.random.default_rng(7)
    A, Bg, Bu = r.standard_normal((3, 4)), r.standard_normal((4, 5)), r.standard_normal((4, 5))
    bg, bu, E = r.standard_normal(5), r.standard_normal(5), r.standard_normal((3, 5))

    def loss(A, Bg, Bu, bg, bu):
        return (E * L.gated(A, Bg, Bu, 1.0, bg, bu, name)[0]).sum()

    _, G, U = L.gated(A, Bg, Bu, 1.0, bg, bu, name)
    dg, du, sg, su = L.gated_grad(E, G, U, name)
    differences(loss, [A, Bg, Bu, bg, bu], [dg @ Bg.T + du @ Bu.T, A.T @ dg, A.T @ du, sg, su],
                atol=1e-5)


@pytest.mark.parametrize("rows", [1, 128])
def test_quantise_blocks_is_the_row_form_of_each_block(rows):
    x = np.random.default_rng(3).standard_normal((200, 300))
    x[5, :128] = 0
    q, s = L.quantise_blocks(x, rows)
    assert s.shape == (-(-200 // rows), 3)
    for i, j in ((0, 0), (1, 2), (-1, 1)):
        i %= len(s)
        at = (slice(i * rows, (i + 1) * rows), slice(128 * j, 128 * j + 128))
        flat, scale = L.quantise_e4m3(x[at].reshape(1, -1))
        np.testing.assert_array_equal(q[at].reshape(1, -1), flat)
        assert s[i, j] == scale[0]
    if rows == 1:
        assert s[5, 0] == 0 and not q[5, :128].any()
    wide = L.spread(s, rows, x.shape)
    assert wide.shape == x.shape and wide[130, 290] == s[130 // rows, 2]
    assert (np.abs(q * wide - x) <= 2.0 ** -4 * np.abs(x) + wide * 2.0 ** -10).all()
