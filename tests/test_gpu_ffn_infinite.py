"""Infinities in the weights and inputs of the gated block's products, whichever way they are computed: an
infinity where the sum of the definition's products has one sign of it, NaN where it has both or meets a zero.

The gradients are tried with projections given by the caller, finite in every feature, so that dz is finite and
the infinities are the products' own."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, P, host  # noqa: F401
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")


def _same_kind(got, ref):
    """Infinite and NaN in the same places, with the same signs; the others within the roundings of dz and the
    result (2^-8 each of the column's largest)."""
    k = lambda t: np.where(np.isfinite(t), 0.0, t)
    np.testing.assert_array_equal(k(got), k(ref))
    fin = np.where(np.isfinite(ref), ref, 0.0)
    assert (np.abs(np.where(np.isfinite(ref), got, 0.0) - fin) <= 2.0 ** -7 * np.abs(fin).max()).all()


def _grads(N, D, F, dt, x, W, z, dh, accumulate=None):
    """(dx, dW) of the library and of the definition."""
    import orthogonal_reparameterized_gb300.poetx as L
    dx = torch.full((N, D), float("nan"), dtype=DT[dt], device=DEV)
    dW = torch.zeros(2 * F, D, dtype=DT[dt], device=DEV) if accumulate is None else accumulate.to(DEV)
    L.poetx_ffn_bwd(x.to(DEV), W.to(DEV), dh.to(DEV), z=z.to(DEV), dx=dx, dW=dW,
                    accumulate=accumulate is not None)
    torch.cuda.synchronize()
    assert L.poetx_get_device_error() == 0
    with np.errstate(invalid="ignore"):
        rdx, rdW = B.ffn_bwd(host(x), host(W), host(dh), B.SILU, host(z))
        if accumulate is not None:
            rdW = rdW + host(accumulate)
    return host(dx), host(dW), rdx, rdW


def _inputs(N, D, F, dt, seed):
    r = np.random.default_rng(seed)
    t = lambda *s: torch.tensor(r.standard_normal(s), dtype=torch.float32).to(DT[dt])
    return t(N, D), t(2 * F, D), t(N, 2 * F), t(N, F)


# every kernel of the gradients: few bf16 rows, up to 128, more; few fp32 rows, more
CASES = [(N, "bf16") for N in (1, 5, 17, 40, 64, 65, 100, 128, 129, 300)] + \
    [(N, "f32") for N in (3, 16, 17, 140)]


@pytest.mark.parametrize("N,dt", CASES)
def test_infinite_weights(P, N, dt):
    """dx = dz W: column 3 of W has an infinity, column 70 two of the same feature's row, column 90 an infinity
    in a feature whose dz is zero (NaN)."""
    D, F = 136, 200
    x, W, z, dh = _inputs(N, D, F, dt, N)
    W[9, 3], W[F + 30, 70], W[31, 90] = INF, -INF, INF
    dh[:, 31] = 0
    dx, dW, rdx, rdW = _grads(N, D, F, dt, x, W, z, dh)
    assert np.isinf(rdx[:, [3, 70]]).all() and np.isnan(rdx[:, 90]).all()
    _same_kind(dx, rdx)
    _same_kind(dW, rdW)


@pytest.mark.parametrize("N,dt", CASES)
@pytest.mark.parametrize("add", [False, True], ids=["set", "add"])
def test_infinite_inputs(P, N, dt, add):
    """dW = dz^T x: x has an infinity in columns 3 and 135; a feature whose dz is zero for that token gets
    NaN there."""
    D, F = 136, 200
    x, W, z, dh = _inputs(N, D, F, dt, N + 1000)
    x[N // 2, 3], x[N - 1, 135] = INF, -INF
    dh[N // 2, 77] = 0
    old = _inputs(2 * F, D, 8, dt, 5)[0] if add else None
    dx, dW, rdx, rdW = _grads(N, D, F, dt, x, W, z, dh, old)
    assert np.isinf(rdW[:, 3]).sum() == 2 * F - 2 and np.isinf(rdW[:, 135]).sum() >= 2 * F - 2
    _same_kind(dx, rdx)
    _same_kind(dW, rdW)


@pytest.mark.parametrize("N,dt", CASES)
def test_nan_among_the_gradients(P, N, dt):
    """A NaN of dz stays in its token's dx and in its feature's dW."""
    D, F = 136, 200
    x, W, z, dh = _inputs(N, D, F, dt, N + 2000)
    dh[N // 2, 40] = float("nan")
    dx, dW, rdx, rdW = _grads(N, D, F, dt, x, W, z, dh)
    _same_kind(dx, rdx)
    _same_kind(dW, rdW)


@pytest.mark.parametrize("N,D,dt", [(1, 264, "bf16"), (40, 264, "bf16"), (300, 264, "bf16"), (3, 264, "f32"),
                                    (20, 264, "f32"), (300, 264, "f32"), (300, 1544, "f32")])
def test_infinity_meets_infinity(P, N, D, dt):
    """x W^T where x and W are infinite in the same place of K, and where one of them alone is."""
    F = 200
    x, W, _, _ = _inputs(N, D, F, dt, 7 * N)
    x[N // 2, 5], W[9, 5], W[F + 12, 5] = INF, INF, -INF
    W[F + 9, 100] = -INF
    z = torch.empty(N, 2 * F, dtype=DT[dt], device=DEV)
    h = torch.empty(N, F, dtype=DT[dt], device=DEV)
    P.poetx_ffn_fwd(x.to(DEV), W.to(DEV), h, z=z)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        ref = host(x) @ host(W).T
    assert ref[N // 2, 9] == INF and ref[N // 2, F + 12] == -INF
    _same_kind(host(z), ref)


@pytest.mark.parametrize("N,D", [(17, 136), (140, 136), (300, 1544)])
def test_infinite_gradient_meets_infinity(P, N, D):
    """fp32 gradients: an infinite dz beside an infinite weight (dx) and an infinite input (dW)."""
    F = 200
    x, W, z, dh = _inputs(N, D, F, "f32", N + 3000)
    dh[N // 2, 40], W[40, 7], W[F + 40, 9], x[N // 2, 30] = INF, INF, -INF, -INF
    dx, dW, rdx, rdW = _grads(N, D, F, "f32", x, W, z, dh)
    assert np.isinf(rdW[[40, F + 40], 30]).all()
    _same_kind(dx, rdx)
    _same_kind(dW, rdW)
