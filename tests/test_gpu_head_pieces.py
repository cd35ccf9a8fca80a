"""Distillation over several pieces of rows, and gradients of up to 128 rows with several vocabulary
tiles per SM, against the fp64 definition."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, P, TOL_BF16_STEP, TOL_F32, dev, host  # noqa: F401
from oracle import head_oracle as H
from test_gpu_head import _ce, _distill, _inputs, _near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_distill_many_rows(P, dt):
    """More rows than a piece takes whatever its bytes: the offsets into the entries, dW over two."""
    N, V, K = 70001, 9, 3
    x, W, _, g = _inputs(N, V, 8, dt, 60)
    r = np.random.default_rng(6)
    idx = r.integers(-1, V, (N, K)).astype(np.int32)
    u = r.uniform(-3, 3, (N, K)).astype(np.float32)
    ref = H.head_distill(host(x), host(W), idx, u, g, 2.0)
    _near(_distill(P, x, W, idx, u, g, 2.0), ref, dt)
    _near(_distill(P, x, W, idx, u, g, 2.0, grads=False), ref, dt)


def test_distill_in_pieces_of_rows(P):
    """More 16-bit values than a piece holds."""
    g = torch.Generator(device=DEV).manual_seed(7)
    N, V, D, K = 9500, 128001, 64, 5
    W = (torch.randn(V, D, generator=g, device=DEV) / 8).bfloat16()
    x = torch.randn(N, D, generator=g, device=DEV).bfloat16()
    idx = torch.randint(0, V, (N, K), generator=g, device=DEV).int()
    idx[::9, 2:] = -1
    idx[5] = -1
    u = 6 * torch.rand(N, K, generator=g, device=DEV)
    dloss = torch.full((N,), 1.0 / N, device=DEV)
    one = P.poetx_head_workspace_bytes(P.BF16, N // 2, D, V, K)
    assert P.poetx_head_workspace_bytes(P.BF16, N, D, V, K) < 1.5 * one  # held in pieces
    got = _distill(P, x, W, idx.cpu().numpy(), u.cpu().numpy(), dloss.cpu().numpy(), 2.0)
    T = 2.0
    z = x.double() @ W.double().T / T
    lse = torch.logsumexp(z, 1)
    there = idx >= 0
    some = there.any(1)
    v = torch.where(there, u.double() / T, torch.full_like(u, -np.inf, dtype=torch.float64))
    q = torch.where(some[:, None], torch.softmax(v, 1), torch.zeros_like(v))
    at = idx.clamp(min=0).long()
    logp = z.gather(1, at) - lse[:, None]
    loss = T * T * torch.where(q > 0, q * (torch.log(q) - logp), torch.zeros_like(q)).sum(1)
    dz = torch.exp(z - lse[:, None])
    dz.scatter_add_(1, at, -q)
    dz *= (dloss.double() * some * T)[:, None]
    for k, ref in (("loss", loss), ("lse", lse), ("dx", dz @ W.double()), ("dW", dz.T @ x.double())):
        tol = TOL_BF16_STEP if k in ("dx", "dW") else TOL_F32
        err = ((got[k].double() - ref).norm() / ref.norm()).item()
        assert err <= tol, (k, err)


@pytest.mark.parametrize("N,V,D", [(1, 60013, 64), (17, 40001, 136), (128, 50257, 72)])
def test_gradients_of_few_rows_and_many_entries(P, N, V, D):
    """More than one vocabulary tile per SM.  Tolerance: the output's rounding (RMS 1.66e-3) and the
    stored exponentials' 2^-11, below 2^-9."""
    x, W, t, g = _inputs(N, V, D, "bf16", N + V)
    got = _ce(P, x, W, t, g)
    ref = H.head_ce(host(x), host(W), t, g)
    for k in ("loss", "lse"):
        assert np.linalg.norm(host(got[k]) - ref[k]) <= TOL_F32 * np.linalg.norm(ref[k]), k
    for k in ("dx", "dW"):
        assert np.linalg.norm(host(got[k]) - ref[k]) <= 2.0 ** -9 * np.linalg.norm(ref[k]), k
