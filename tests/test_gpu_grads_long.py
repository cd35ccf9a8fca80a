"""The global gradient norm of long tensors: its error does not grow with the number of elements.

Tolerance: sixteen squares are added in fp32 (nine roundings of 2^-24 at most in a row, for terms of one
sign relative to the sum), their sums without loss, the root halves what is left and its rounding is one
more: 5.5 x 2^-24, below 2^-21.  Equal terms round the same way every time, so that a sum kept in fp32
drifts; random ones hide it."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, P  # noqa: F401

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -21


def _norm(P, ts):
    n = torch.full((1,), float("nan"), device=DEV)
    P.poetx_grad_norm(ts, n)
    return float(n)


def _exact(t):
    """In 64 bits, a piece at a time."""
    return float(sum((p.double() ** 2).sum() for p in t.split(1 << 24))) ** 0.5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_norm_of_equal_values(P, dtype):
    """Hundreds of adds per thread of the whole GPU."""
    n = (1 << 29) + 77 if dtype is torch.bfloat16 else (1 << 28) + 77
    x = torch.empty(n, dtype=dtype, device=DEV)
    off = {}
    for c in (0.3, 0.1, 0.7, 1.0 / 3, 1.9, 1e-3):
        x.fill_(c)
        off[c] = _norm(P, [x]) / (float(x[0]) * np.sqrt(n)) - 1
    assert max(map(abs, off.values())) <= TOL, off


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_norm_of_many_random_values(P, dtype):
    g = torch.Generator(device=DEV).manual_seed(5)
    x = (torch.randn((1 << 27) + 5, generator=g, device=DEV) * 3e-3).to(dtype)
    y = (torch.randn(1000003, generator=g, device=DEV) * 0.2).to(dtype)
    for ts in ([x], [y, x, y[:8]], [x[:1 << 20]] * 300):
        ref = sum(_exact(t) ** 2 for t in ts) ** 0.5
        assert abs(_norm(P, ts) / ref - 1) <= TOL


def test_norm_of_values_of_many_sizes(P):
    """Magnitudes from 2^-60 to 2^60 beside each other: what one sum takes up in 64 bits and the other in fp32
    add up."""
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(1 << 22, generator=g, device=DEV)
    for lo, hi in ((-60, -40), (-20, 20), (40, 60), (-60, 60)):
        t = x * torch.exp2(torch.randint(lo, hi, x.shape, generator=g, device=DEV).float())
        assert abs(_norm(P, [t]) / _exact(t) - 1) <= TOL, (lo, hi)
