"""Refusals of the layer norm and head entry points: host-side checks, before any launch (run
without a GPU; the pointers are never dereferenced)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def P():
    from orthogonal_reparameterized_gb300 import build
    build.build()
    import orthogonal_reparameterized_gb300.poetx as P
    P.lib()
    return P


ARG, SHAPE, DTYPE, ALIGN, WORKSPACE = 1, 2, 3, 4, 5
OK = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4100)


def _fwd(P, **kw):
    a = dict(dt=P.BF16, x=OK, N=4, D=64, gamma=OK, beta=OK, eps=1e-5, y=OK, mean=OK, rstd=OK)
    a.update(kw)
    return P.lib().poetx_layernorm_fwd(*a.values(), None)


def _bwd(P, **kw):
    a = dict(dt=P.BF16, x=OK, dy=OK, N=4, D=64, gamma=OK, mean=OK, rstd=OK, dx=OK, dgamma=OK,
             dbeta=OK, accumulate=0, ws=OK, ws_bytes=1 << 30)
    a.update(kw)
    return P.lib().poetx_layernorm_bwd(*a.values(), None)


def _ce(P, **kw):
    a = dict(dt=P.BF16, x=OK, N=4, D=64, W=OK, V=100, target=OK, z=0.0, dloss=OK, loss=OK, lse=OK,
             dx=OK, dW=OK, accumulate=0, ws=OK, ws_bytes=1 << 34)
    a.update(kw)
    return P.lib().poetx_head_ce(*a.values(), None)


def _distill(P, **kw):
    a = dict(dt=P.BF16, x=OK, N=4, D=64, W=OK, V=100, idx=OK, logit=OK, K=5, T=1.0, dloss=OK,
             loss=OK, lse=OK, dx=OK, dW=OK, accumulate=0, ws=OK, ws_bytes=1 << 34)
    a.update(kw)
    return P.lib().poetx_head_distill(*a.values(), None)


@pytest.mark.parametrize("kw,st", [
    (dict(N=-1), ARG), (dict(D=0), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(dt=2), DTYPE), (dict(dt=9), DTYPE), (dict(x=None), ARG), (dict(y=None), ARG),
    (dict(x=ODD), ALIGN), (dict(y=ODD), ALIGN), (dict(gamma=ODD), ALIGN), (dict(rstd=ODD), ALIGN),
    (dict(N=0), 0)])
def test_layernorm_fwd_refusals(P, kw, st):
    assert _fwd(P, **kw) == st


@pytest.mark.parametrize("kw,st", [
    (dict(N=-1), ARG), (dict(D=0), ARG), (dict(dt=2), DTYPE), (dict(x=None), ARG),
    (dict(dy=None), ARG), (dict(mean=None), ARG), (dict(rstd=None), ARG), (dict(dx=None), ARG),
    (dict(ws=None), ARG), (dict(ws_bytes=64), WORKSPACE), (dict(dy=ODD), ALIGN),
    (dict(dgamma=ODD), ALIGN), (dict(ws=ODD), ALIGN)])
def test_layernorm_bwd_refusals(P, kw, st):
    assert _bwd(P, **kw) == st


HEAD = [
    (dict(N=-1), ARG), (dict(dt=2), DTYPE), (dict(D=60), SHAPE), (dict(D=0), SHAPE),
    (dict(D=131080), SHAPE), (dict(V=0), SHAPE), (dict(V=4194305), SHAPE), (dict(x=None), ARG),
    (dict(W=None), ARG), (dict(loss=None), ARG), (dict(dloss=None), ARG), (dict(ws=None), ARG),
    (dict(ws_bytes=1024), WORKSPACE), (dict(x=ODD), ALIGN), (dict(W=ODD), ALIGN),
    (dict(dx=ODD), ALIGN), (dict(dW=ODD), ALIGN), (dict(loss=ODD), ALIGN), (dict(ws=ODD), ALIGN)]


@pytest.mark.parametrize("kw,st", HEAD + [
    (dict(target=None), ARG), (dict(target=ODD), ALIGN), (dict(z=-0.1), ARG),
    (dict(z=float("nan")), ARG)])
def test_ce_refusals(P, kw, st):
    assert _ce(P, **kw) == st


@pytest.mark.parametrize("kw,st", HEAD + [
    (dict(K=0), SHAPE), (dict(K=1025), SHAPE), (dict(T=0.0), ARG), (dict(T=-1.0), ARG),
    (dict(T=float("nan")), ARG), (dict(idx=None), ARG), (dict(logit=None), ARG),
    (dict(logit=ODD), ALIGN)])
def test_distill_refusals(P, kw, st):
    assert _distill(P, **kw) == st


def test_workspace_sizes(P):
    b = P.poetx_head_workspace_bytes
    assert b(P.BF16, 4096, 2048, 32000, 1, True, True) >= 4096 * 32000 * 2
    # the loss alone holds no value per logit, only two per 128 of them
    assert b(P.BF16, 4096, 2048, 32000, 1, False, False) < 4096 * 32000 // 4
    # many rows go in pieces: the 16-bit values held stay near 1 GiB
    assert b(P.BF16, 1 << 20, 64, 128000, 1, True, False) < 3 << 30
    for bad in ((P.I8, 4, 64, 100, 1), (P.BF16, -1, 64, 100, 1), (P.BF16, 4, 65, 100, 1),
                (P.BF16, 4, 64, 0, 1), (P.BF16, 4, 64, 100, 0), (P.BF16, 4, 64, 100, 2000)):
        assert b(*bad) == 0, bad
    n = P.poetx_layernorm_bwd_workspace_bytes
    assert n(P.BF16, 8192, 4096) >= 2 * 4096 * 4
    assert n(P.I8, 8, 8) == n(P.BF16, -1, 8) == n(P.BF16, 8, 0) == 0


def test_binding_checks_shapes(P):
    x, W = torch.zeros(4, 64), torch.zeros(100, 64)
    t, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(ValueError, match="target"):
        P.poetx_head_ce(x, W, t.long(), f)
    with pytest.raises(ValueError, match="W must be"):
        P.poetx_head_ce(x, W[:, :32], t, f)
    with pytest.raises(ValueError, match="loss"):
        P.poetx_head_ce(x, W, t, f[:3])
    with pytest.raises(ValueError, match="t_logit"):
        P.poetx_head_distill(x, W, t[:, None], f, f)
    with pytest.raises(ValueError, match="y must be"):
        P.poetx_layernorm_fwd(x, x.bfloat16())
    with pytest.raises(ValueError, match="gamma"):
        P.poetx_layernorm_fwd(x, x.clone(), gamma=torch.zeros(63))
    with pytest.raises(ValueError, match="rstd"):
        P.poetx_layernorm_bwd(x, x, f, f[:2], x.clone())
    with pytest.raises(ValueError, match="CUDA"):
        P.poetx_layernorm_fwd(x, x.clone())
