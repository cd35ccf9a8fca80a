"""The fp64 definitions of the block's operators: their gradients against differences, and what
must hold of them by themselves."""
import numpy as np
import pytest

from oracle import block_oracle as B


def _differences(f, x, dy, h=1e-6):
    """The gradient of sum(f(x) dy) by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = ((f(up) - f(down)) * dy).sum() / (2 * h)
    return g


@pytest.mark.parametrize("act", [B.SILU, B.GELU])
def test_ffn_gradients(act):
    r = np.random.default_rng(1)
    x, W, dh = r.standard_normal((3, 4)), r.standard_normal((10, 4)), r.standard_normal((3, 5))
    dx, dW = B.ffn_bwd(x, W, dh, act)
    # central differences of values near 1 with a step of 1e-6: 1e-16 / 1e-6 and the step's square
    np.testing.assert_allclose(dx, _differences(lambda t: B.ffn(t, W, act)[0], x, dh), atol=1e-8)
    np.testing.assert_allclose(dW, _differences(lambda t: B.ffn(x, t, act)[0], W, dh), atol=1e-8)
    z = B.ffn(x, W, act)[1]
    np.testing.assert_array_equal(B.ffn_bwd(x, W, dh, act, z)[1], dW)


def test_activation_values():
    g = np.array([0.0, 1.0, -1.0, 30.0, -30.0])
    np.testing.assert_allclose(B.activation(g, B.SILU)[0], g / (1 + np.exp(-g)), rtol=1e-15)
    # the tanh form is the erf form to about 1e-3
    from math import erf, sqrt
    ref = [0.5 * v * (1 + erf(v / sqrt(2))) for v in g]
    np.testing.assert_allclose(B.activation(g, B.GELU)[0], ref, atol=1e-3)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rot", [4, 8])
def test_rope_gradients(interleaved, norm, rot):
    r = np.random.default_rng(2)
    x, dy = r.standard_normal((3, 2, 8)), r.standard_normal((3, 2, 8))
    gamma = 1 + 0.3 * r.standard_normal(8)
    pos = r.integers(-50, 50, (2, 3))
    freq = 10.0 ** -np.arange(rot // 2)
    axis = np.arange(rot // 2) % 2
    kw = dict(axis=axis, interleaved=interleaved, norm=norm, eps=1e-3)
    dx, dgamma = B.qk_rope_bwd(x, dy, pos, freq, gamma=gamma, **kw)
    np.testing.assert_allclose(
        dx, _differences(lambda t: B.qk_rope(t, pos, freq, gamma=gamma, **kw), x, dy), atol=1e-8)
    if norm:
        np.testing.assert_allclose(
            dgamma, _differences(lambda t: B.qk_rope(x, pos, freq, gamma=t, **kw), gamma, dy),
            atol=1e-8)


def test_rope_keeps_lengths_and_depends_on_distances():
    r = np.random.default_rng(3)
    x = r.standard_normal((2, 1, 8))
    freq = np.array([1.0, 0.3, 0.1, 0.01])
    y = B.qk_rope(x, np.array([[7, 100]]), freq, norm=False)
    np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-14)
    z = B.qk_rope(x, np.array([[12, 105]]), freq, norm=False)
    np.testing.assert_allclose(y[0, 0] @ y[1, 0], z[0, 0] @ z[1, 0], rtol=1e-12)


def test_norm_and_factor():
    assert B.grad_norm([np.array([3.0]), np.array([[4.0]])]) == 5.0
    assert B.clip_factor(0.0, 1.0) == 1.0
    assert B.clip_factor(0.5, 1.0) == 1.0
    assert abs(B.clip_factor(4.0, 1.0) - 0.25) < 1e-6
