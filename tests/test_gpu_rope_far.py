"""The rotation's angles over all positions and frequencies up to 2 pi.

Tolerance of an output a cos t - b sin t in fp32, times |a| + |b|: t is off by 2^-26 turns (its rounding to
fp32) and 2^-32 (its reduction), 9.6e-8; sine and cosine by one unit in the last place, 6e-8; the product and
the sum by 2^-24 each: 2.8e-7, below 2^-21.5.  A reduction that loses 2^-22 turns is off by 1.5e-6."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, P, dev, host  # noqa: F401
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -21.5


def _frequencies(kind, half, r):
    if kind == "usual":
        return (10000.0 ** (-np.arange(half) / half)).astype(np.float32)
    sign = np.where(r.random(half) < 0.5, -1.0, 1.0)
    f = (sign * r.uniform(3.0, 6.283, half)).astype(np.float32)
    f[:2] = (6.2831850, -6.2831850)
    return f


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("kind", ["usual", "to_2_pi"])
def test_rope_angles_of_far_positions(P, kind, interleaved):
    N, dh = 1500, 64
    r = np.random.default_rng(3)
    x = torch.tensor(r.standard_normal((N, 1, dh)), dtype=torch.float32)
    pos = r.integers(-2 ** 31, 2 ** 31, (1, N)).astype(np.int32)
    pos[0, :5] = (2 ** 31 - 1, -2 ** 31, 0, 1, -1)
    pos[0, 5:300] = r.integers(-2 ** 20, 2 ** 20, 295)
    freq = _frequencies(kind, dh // 2, r)
    first, second = B._pairs(dh, interleaved)
    xh = host(x)
    size = np.empty_like(xh)
    size[..., first] = size[..., second] = np.abs(xh[..., first]) + np.abs(xh[..., second])
    xd, y = x.to(DEV), torch.empty_like(x, device=DEV)
    args = dev(pos, torch.int32), dev(freq, torch.float32)
    P.poetx_qk_rope_fwd(xd, None, *args, y, None, interleaved=interleaved, norm=False)
    ref = B.qk_rope(xh, pos, freq, interleaved=interleaved, norm=False)
    assert (np.abs(host(y) - ref) / size).max() <= TOL
    P.poetx_qk_rope_bwd(xd, None, xd, None, *args, y, None, interleaved=interleaved, norm=False)
    ref, _ = B.qk_rope_bwd(xh, xh, pos, freq, interleaved=interleaved, norm=False)
    assert (np.abs(host(y) - ref) / size).max() <= TOL
