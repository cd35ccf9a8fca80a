"""CPU pins of the fp64 definitions of layer norm, the head's cross entropy and distillation:
closed forms, and every gradient against central differences of its own loss."""
import numpy as np
import pytest

from oracle import head_oracle as H


def _rng(seed):
    return np.random.default_rng(seed)


def _central(f, a, step=1e-6):
    """Gradient of the scalar f with respect to the array a, by central differences (error
    O(step^2) plus 1e-16 / step = 1e-10 of f)."""
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + step
        up = f()
        a[i] = keep - step
        down = f()
        a[i] = keep
        g[i] = (up - down) / (2 * step)
    return g


def test_layernorm_closed_forms():
    y, mean, rstd = H.layernorm(np.array([[1.0, 3.0]]), eps=0.0)
    np.testing.assert_allclose(y, [[-1.0, 1.0]])
    assert mean[0] == 2.0 and rstd[0] == 1.0
    y, _, rstd = H.layernorm(np.array([[5.0]]), beta=np.array([0.25]), eps=0.01)
    assert y[0, 0] == 0.25 and rstd[0] == pytest.approx(10.0)


@pytest.mark.parametrize("affine", [False, True])
def test_layernorm_gradient_is_the_difference(affine):
    r = _rng(1)
    x, w = r.standard_normal((3, 5)), r.standard_normal((3, 5))
    gamma = r.standard_normal(5) if affine else None
    beta = r.standard_normal(5) if affine else None
    f = lambda: float((H.layernorm(x, gamma, beta)[0] * w).sum())
    dx, dgamma, dbeta = H.layernorm_bwd(x, w, gamma)
    np.testing.assert_allclose(dx, _central(f, x), atol=1e-7)
    if affine:
        np.testing.assert_allclose(dgamma, _central(f, gamma), atol=1e-7)
        np.testing.assert_allclose(dbeta, _central(f, beta), atol=1e-7)


def test_ce_closed_form():
    # two equal logits: loss ln 2, dz = (1/2 - 1, 1/2)
    o = H.head_ce(np.array([[2.0]]), np.array([[1.0], [1.0]]), np.array([0]), np.ones(1))
    assert o["loss"][0] == pytest.approx(np.log(2))
    assert o["dx"][0, 0] == pytest.approx(0.0)
    np.testing.assert_allclose(o["dW"][:, 0], [-1.0, 1.0])


@pytest.mark.parametrize("z_loss", [0.0, 0.3])
def test_ce_gradient_is_the_difference(z_loss):
    r = _rng(2)
    x, W = r.standard_normal((4, 3)), r.standard_normal((6, 3))
    t, g = np.array([5, -100, 0, 2]), r.standard_normal(4)
    f = lambda: float((H.head_ce(x, W, t, z_loss=z_loss)["loss"] * g).sum())
    o = H.head_ce(x, W, t, g, z_loss)
    np.testing.assert_allclose(o["dx"], _central(f, x), atol=1e-7)
    np.testing.assert_allclose(o["dW"], _central(f, W), atol=1e-7)
    assert o["loss"][1] == 0 and not o["dx"][1].any()


@pytest.mark.parametrize("T", [1.0, 2.5])
def test_distill_gradient_is_the_difference(T):
    r = _rng(3)
    x, W = r.standard_normal((4, 3)), r.standard_normal((7, 3))
    idx = np.array([[0, 3, 6], [2, -1, 5], [-1, -1, -1], [4, 4, 1]])  # absent, empty, repeated
    u, g = r.standard_normal((4, 3)), r.standard_normal(4)
    f = lambda: float((H.head_distill(x, W, idx, u, temperature=T)["loss"] * g).sum())
    o = H.head_distill(x, W, idx, u, g, T)
    np.testing.assert_allclose(o["dx"], _central(f, x), atol=1e-7)
    np.testing.assert_allclose(o["dW"], _central(f, W), atol=1e-7)
    assert o["loss"][2] == 0 and not o["dx"][2].any()


def test_distill_with_one_entry_is_cross_entropy():
    r = _rng(4)
    x, W, t, g = r.standard_normal((5, 4)), r.standard_normal((9, 4)), r.integers(0, 9, 5), np.ones(5)
    a = H.head_ce(x, W, t, g)
    b = H.head_distill(x, W, t[:, None], r.standard_normal((5, 1)), g)
    for k in a:
        np.testing.assert_allclose(a[k], b[k], atol=1e-12)


def test_distill_against_the_whole_vocabulary_vanishes_at_the_student():
    r = _rng(5)
    x, W = r.standard_normal((3, 4)), r.standard_normal((6, 4))
    idx = np.tile(np.arange(6), (3, 1))
    o = H.head_distill(x, W, idx, x @ W.T, np.ones(3), 2.0)
    for k in ("loss", "dx", "dW"):
        np.testing.assert_allclose(o[k], 0, atol=1e-12)
