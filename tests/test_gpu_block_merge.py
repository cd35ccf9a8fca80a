"""The gated feed-forward block over the merged weights of a POET-X gate and up layer: what the two layers and the
gated product between them and the down layer compute, in one call (a trained block being served).

Tolerance: fp32 sums on both sides, a merge, a product and the gated product behind it: 10 TOL_F32; in bf16 the
weights' rounding, x's and the result's: three of 2^-8 at most, in a norm over all elements."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import DEV, P, TOL_F32, dev, host  # noqa: F401
from oracle import block_oracle as B
from test_gpu_block_chain import Layer

pytestmark = pytest.mark.gpu


def _merged(P, layers, n, m):
    """[2 n, m] fp32: the layers' current maps one below the other."""
    W = torch.empty(2 * n, m, device=DEV)
    for half, L in zip(W.split(n), layers):
        P.poetx_merge_reinit(L.L, half, P.workspace(P.poetx_merge_reinit_workspace_bytes(L.L), DEV))
    return W


@pytest.mark.parametrize("N", [1, 5, 70, 200])
def test_merged_gate_and_up(P, N):
    D, F, b = 128, 192, 32
    gate, up = (Layer(P, D, F, b, N, 60 + i) for i in range(2))
    r = np.random.default_rng(N)
    x, dh = (dev(r.standard_normal(s), torch.float32) for s in ((N, D), (N, F)))
    # as it is trained: two layers and the product
    g, u = gate.forward(x), up.forward(x)
    h = torch.empty(N, F, device=DEV)
    P.poetx_glu_fwd(g, u, h)
    dg, du = torch.empty_like(g), torch.empty_like(u)
    P.poetx_glu_bwd(g, u, dh, dg, du)
    dx = gate.backward(dg) + up.backward(du)
    # as it is served (or trained on with whole weights)
    W = _merged(P, (gate, up), F, D)
    h2, z, dx2 = torch.empty(N, F, device=DEV), torch.empty(N, 2 * F, device=DEV), torch.empty(N, D, device=DEV)
    P.poetx_ffn_fwd(x, W, h2, z=z)
    P.poetx_ffn_bwd(x, W, dh, z=z, dx=dx2)
    torch.cuda.synchronize()
    assert P.poetx_get_device_error() == 0
    ref = B.glu(*(L.oracle(host(x))["y"] for L in (gate, up)), B.SILU)
    for a in (h, h2):
        assert O.rel_fro(host(a), ref) <= 10 * TOL_F32
    assert O.rel_fro(host(z), host(torch.cat([g, u], 1))) <= 10 * TOL_F32
    assert O.rel_fro(host(dx2), host(dx)) <= 10 * TOL_F32
    h16 = torch.empty(N, F, device=DEV).bfloat16()
    P.poetx_ffn_fwd(x.bfloat16(), W.bfloat16(), h16)
    assert O.rel_fro(host(h16), ref) <= 3 * 2.0 ** -8
