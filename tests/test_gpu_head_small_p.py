"""Gradients element by element against the fp64 definition, down to probabilities far below their
neighbours'.

Bounds (u = 2^-8, a bf16 rounding; A = |dz|^T |x| or |dz| |W|, the products' absolute sums).  The
stored exponentials carry 11 bits (2^-11 of each dz), dz is rounded to bf16 over more than 128 rows
(u) and to two bf16 pieces over fewer (2^-16), the fp32 sums add less than 2^-13 of A, and the result
is rounded once: (u + 2^-11 + 2^-13) A, or (2^-11 + 2^-16 + 2^-13) A, plus u |ref|."""
import numpy as np
import pytest

from gpu_util import P, host  # noqa: F401
from test_gpu_head import _ce, _distill, _inputs

import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def _dz(x, W, t, g):
    z = host(x) @ host(W).T
    z -= z.max(axis=1, keepdims=True)
    p = np.exp(z)
    p /= p.sum(axis=1, keepdims=True)
    rows = np.nonzero(t >= 0)[0]
    p[rows, t[rows]] -= 1
    p[t < 0] = 0
    return p * g.astype(np.float64)[:, None]


def _check(got, x, W, dz, N):
    rel = 2.0 ** -11 + 2.0 ** -13 + (2.0 ** -16 if N <= 128 else U)
    x, W = host(x), host(W)
    for k, a, b in (("dx", dz, W), ("dW", dz.T, x)):
        ref, mag = a @ b, np.abs(a) @ np.abs(b)
        over = np.abs(host(got[k]) - ref) - (rel * mag + U * np.abs(ref))
        at = np.unravel_index(over.argmax(), over.shape)
        assert over[at] <= 1e-37, (k, at, host(got[k])[at], ref[at], mag[at])


def _ladder(N, V, seed):
    """Logits of 0 in every 16th column and 8 to 36 nats below it in the others, in every row."""
    r = np.random.default_rng(seed)
    W, x = np.zeros((V, 64)), r.standard_normal((N, 64))
    W[:, 0] = -r.uniform(8, 36, V)
    W[::16, 0] = 0
    x[:, 0] = 1
    t = (16 * r.integers(0, V // 16, N)).astype(np.int32)
    g = (r.uniform(0.5, 1.5, N) / N).astype(np.float32)
    return torch.tensor(x).bfloat16(), torch.tensor(W).bfloat16(), t, g


# the product of few rows (tiles of 16 and of 128 vocabulary rows), the one of many, with a tail
@pytest.mark.parametrize("N,V", [(1, 512), (40, 1024), (128, 20000), (129, 1040), (300, 4000)])
def test_gradients_far_below_the_group_maximum(P, N, V):
    x, W, t, g = _ladder(N, V, N)
    dz = _dz(x, W, t, g)
    _check(_ce(P, x, W, t, g), x, W, dz, N)
    # a teacher that knows one entry: the same gradients
    _check(_distill(P, x, W, t[:, None], np.zeros((N, 1), np.float32), g), x, W, dz, N)


@pytest.mark.parametrize("N,V,D", [(5, 300, 72), (64, 5003, 264), (128, 40001, 128), (129, 257, 200),
                                   (301, 5003, 136), (700, 3001, 520)])
def test_gradients_element_by_element(P, N, V, D):
    x, W, t, g = _inputs(N, V, D, "bf16", 3 * N + V)
    t[::7] = -1
    _check(_ce(P, x, W, t, g), x, W, _dz(x, W, t, g), N)


def test_gradients_of_large_logits(P):
    """Logits to some ten thousand, where a group's maximum is rounded by 2^-10: the largest stored
    exponential is then not exactly 1."""
    x, W, t, g = _inputs(200, 900, 64, "bf16", 50)
    x = (x.float() * 4000).bfloat16()
    got = _ce(P, x, W, t, g)
    assert all(torch.isfinite(got[k]).all() for k in got)
    # p is 0 or 1 here but for ties: the bound on dz is the fp32 logits' own error
    dz = _dz(x, W, t, g)
    assert np.abs(host(got["dW"]) - dz.T @ host(x)).max() <= 2e-2 * (np.abs(dz).T @ np.abs(host(x))).max()
