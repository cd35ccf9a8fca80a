"""The upstream gradient of a row that gives no gradient does not matter, whatever stands there."""
import numpy as np
import pytest
import torch

from gpu_util import P, host  # noqa: F401
from test_gpu_head import _ce, _distill, _inputs

pytestmark = pytest.mark.gpu

ROWS = [("bf16", 40), ("bf16", 128), ("bf16", 301), ("f32", 301)]
JUNK = [1e38, -3e38, float("inf"), float("nan"), 1.0]


def _same(a, b):
    for k in a:
        assert torch.equal(a[k].nan_to_num(7.0), b[k].nan_to_num(7.0)), k


@pytest.mark.parametrize("dt,N", ROWS)
@pytest.mark.parametrize("junk", JUNK)
def test_ce(P, dt, N, junk):
    x, W, t, g = _inputs(N, 600, 64, dt, 40)
    t[::3] = -100
    t[1], t[N - 2] = 600, 2 ** 31 - 1  # beyond the vocabulary: loss NaN, gradient 0
    off = (t < 0) | (t >= 600)
    g[off] = 0
    ref = _ce(P, x, W, t, g)
    assert np.abs(host(ref["dW"])).max() > 1e-4 and not host(ref["dx"])[off].any()
    g[off] = junk
    _same(ref, _ce(P, x, W, t, g))


@pytest.mark.parametrize("dt,N", ROWS)
@pytest.mark.parametrize("junk", JUNK)
def test_distill(P, dt, N, junk):
    x, W, _, g = _inputs(N, 600, 64, dt, 41)
    r = np.random.default_rng(3)
    idx = np.stack([r.permutation(600)[:5] for _ in range(N)]).astype(np.int32)
    u = r.uniform(-3, 6, (N, 5)).astype(np.float32)
    idx[::3] = -1
    u[1] = -np.inf
    u[2, :3], idx[2, 3:] = -np.inf, -5
    idx[4, 2] = 600
    off = np.zeros(N, bool)
    off[::3] = off[[1, 2, 4]] = True
    g[off] = 0
    ref = _distill(P, x, W, idx, u, g, 2.0)
    assert np.abs(host(ref["dW"])).max() > 1e-4 and not host(ref["dx"])[off].any()
    g[off] = junk
    _same(ref, _distill(P, x, W, idx, u, g, 2.0))
