"""The training head's operators together: norm -> head -> norm's backward against the fp64
definitions, and the example's training steps."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle as O
from conftest import ROOT
from gpu_util import DEV, P, TOL_F32, dev, host  # noqa: F401
from oracle import head_oracle as H

pytestmark = pytest.mark.gpu


def test_norm_head_chain_fp32(P):
    """fp32 throughout: the chain's gradients to a few TOL_F32 (three products, a norm and its
    backward one after the other)."""
    N, V, D = 130, 1003, 264
    r = np.random.default_rng(21)
    x = r.standard_normal((N, D)).astype(np.float32) * 3 + 1
    gamma, beta = (1 + 0.1 * r.standard_normal(D)).astype(np.float32), \
        (0.1 * r.standard_normal(D)).astype(np.float32)
    W = (r.standard_normal((V, D)) / np.sqrt(D)).astype(np.float32)
    t = r.integers(0, V, N).astype(np.int32)
    t[5] = -1
    g = np.full(N, 1 / (N - 1), np.float32)
    f32 = lambda *s: torch.empty(*s, device=DEV)
    xd, gd, bd, Wd = (dev(a, torch.float32) for a in (x, gamma, beta, W))
    h, dh, dx, mean, rstd, loss, dW = f32(N, D), f32(N, D), f32(N, D), f32(N), f32(N), f32(N), f32(V, D)
    dgamma, dbeta = f32(D), f32(D)
    P.poetx_layernorm_fwd(xd, h, gamma=gd, beta=bd, mean=mean, rstd=rstd)
    P.poetx_head_ce(h, Wd, dev(t, torch.int32), loss, dloss=dev(g, torch.float32), dx=dh, dW=dW)
    P.poetx_layernorm_bwd(xd, dh, mean, rstd, dx, gamma=gd, dgamma=dgamma, dbeta=dbeta)
    torch.cuda.synchronize()
    y, _, _ = H.layernorm(x, gamma, beta)
    head = H.head_ce(y, W, t, g)
    rdx, rdg, rdb = H.layernorm_bwd(x, head["dx"], gamma)
    for got, ref in ((loss, head["loss"]), (dW, head["dW"]), (dx, rdx), (dgamma, rdg), (dbeta, rdb)):
        assert O.rel_fro(host(got), ref) <= 3 * TOL_F32


def test_example_learns(P):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_head
    finally:
        sys.path.pop(0)
    ce, kd = train_head.train(steps=12, tokens=256, width=256, vocab=1001)
    assert np.isfinite(ce + kd).all()
    assert ce[-1] < 0.8 * ce[0] and kd[-1] < 0.8 * kd[0], (ce, kd)
