"""The block's operators together, as a training step uses them, against the fp64 definitions: norm ->
POET-X query and key layers -> norms and rotation, and norm -> POET-X gate and up layers -> gated product ->
POET-X down layer, their way back, the gradients' norm and the clipped update; norm -> gated feed-forward
block -> head; and the example's steps."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle as O
from conftest import ROOT
from gpu_util import DEV, P, TOL_F32, dev, host  # noqa: F401
from oracle import block_oracle as B
from oracle import head_oracle as H

pytestmark = pytest.mark.gpu


class Layer:
    """An fp32 POET-X layer and its inputs for the oracle."""

    def __init__(self, P, m, n, b, N, seed):
        from orthogonal_reparameterized_gb300 import inputs
        self.P, self.N, self.b = P, N, b
        self.inp = inputs.small_layer_inputs(seed, m, n, b, N, act="f32", wdt="f32", q_std=0.02)
        W0 = dev(self.inp["W0"], torch.float32)
        self.pm, self.pn = (dev(self.inp[k], torch.int32) for k in ("perm_m", "perm_n"))
        self.Wp = torch.empty_like(W0)
        P.poetx_merge_perm(W0, self.pn, self.pm, self.Wp)
        self.q = [dev(self.inp[k], torch.float32) for k in ("q_R", "q_P")]
        self.dq = [torch.empty_like(t) for t in self.q]
        self.L = P.make_layer(m, n, b, P.F32, P.F32, P.FAST, self.pm, self.pn, self.Wp, *self.q)
        self.saved = P.workspace(P.poetx_layer_saved_bytes(self.L, N), DEV)
        self.ws = P.workspace(max(P.poetx_layer_workspace_bytes(self.L, N, k) for k in (0, 1)), DEV)
        self.y, self.dx = torch.empty(N, n, device=DEV), torch.empty(N, m, device=DEV)

    def forward(self, x):
        self.x = x
        self.P.poetx_layer_fwd(self.L, x, self.y, self.saved, self.ws)
        return self.y

    def backward(self, dy):
        self.P.poetx_layer_bwd(self.L, self.x, dy, self.saved, self.dx, *self.dq, self.ws)
        return self.dx

    def oracle(self, x, dy=None):
        i = self.inp
        return O.poetx_layer(x, np.zeros((self.N, i["W0"].shape[0])) if dy is None else dy, i["W0"],
                             i["perm_m"], i["perm_n"], i["q_R"], i["q_P"], self.b)


def _f32(*shape):
    return torch.empty(*shape, device=DEV)


def test_poetx_block_chain_fp32(P):
    """Tolerance: a handful of TOL_F32 (a norm, two layers and two products one after the other)."""
    N, D, F, b, heads, dh = 70, 128, 192, 32, 4, 32
    r = np.random.default_rng(31)
    x = (r.standard_normal((N, D)) * 2 + 0.5).astype(np.float32)
    gamma = (1 + 0.1 * r.standard_normal(D)).astype(np.float32)
    gq, gk = ((1 + 0.1 * r.standard_normal(dh)).astype(np.float32) for _ in range(2))
    pos = np.stack([np.arange(N) + 5000, np.arange(N) // 8]).astype(np.int32)
    freq = (10000.0 ** (-np.arange(dh // 2) / (dh // 2))).astype(np.float32)
    axis = (np.arange(dh // 2) % 2).astype(np.int32)
    up = {k: r.standard_normal((N, heads, dh)).astype(np.float32) for k in "qk"}
    dy = r.standard_normal((N, D)).astype(np.float32)
    Lq, Lk, Lg, Lu = (Layer(P, D, n, b, N, 40 + i) for i, n in enumerate((D, D, F, F)))
    Ld = Layer(P, F, D, b, N, 44)
    # the library
    xd, gd = dev(x, torch.float32), dev(gamma, torch.float32)
    h, mean, rstd = _f32(N, D), _f32(N), _f32(N)
    P.poetx_layernorm_fwd(xd, h, gamma=gd, mean=mean, rstd=rstd)
    q, k = (L.forward(h).view(N, heads, dh) for L in (Lq, Lk))
    kw = dict(axis=dev(axis, torch.int32), gamma_q=dev(gq, torch.float32), gamma_k=dev(gk, torch.float32))
    pd, fd = dev(pos, torch.int32), dev(freq, torch.float32)
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    P.poetx_qk_rope_fwd(q, k, pd, fd, qr, kr, **kw)
    g, u = Lg.forward(h), Lu.forward(h)
    a = _f32(N, F)
    P.poetx_glu_fwd(g, u, a)
    y = Ld.forward(a)
    da = Ld.backward(dev(dy, torch.float32))
    dg, du = torch.empty_like(g), torch.empty_like(u)
    P.poetx_glu_bwd(g, u, da, dg, du)
    dq, dk, dgq, dgk = torch.empty_like(q), torch.empty_like(k), _f32(dh), _f32(dh)
    P.poetx_qk_rope_bwd(q, k, dev(up["q"], torch.float32), dev(up["k"], torch.float32), pd, fd, dq, dk,
                        dgamma_q=dgq, dgamma_k=dgk, **kw)
    dh_ = Lg.backward(dg) + Lu.backward(du) + Lq.backward(dq.view(N, D)) + Lk.backward(dk.view(N, D))
    dx, dgamma = _f32(N, D), _f32(D)
    P.poetx_layernorm_bwd(xd, dh_, mean, rstd, dx, gamma=gd, dgamma=dgamma)
    layers = [Lq, Lk, Lg, Lu, Ld]
    grads = [t for L in layers for t in L.dq] + [dgamma, dgq, dgk]
    norm = _f32(1)
    P.poetx_grad_norm(grads, norm)
    # the definitions
    h64, _, _ = H.layernorm(x, gamma)
    o = dict(axis=axis)
    q64, k64 = (L.oracle(h64)["y"].reshape(N, heads, dh) for L in (Lq, Lk))
    g64, u64 = Lg.oracle(h64)["y"], Lu.oracle(h64)["y"]
    d = {Ld: Ld.oracle(B.glu(g64, u64, B.SILU), dy)}
    dg64, du64 = B.glu_bwd(g64, u64, d[Ld]["dx"], B.SILU)
    dq64, dgq64 = B.qk_rope_bwd(q64, up["q"], pos, freq, gamma=gq, **o)
    dk64, dgk64 = B.qk_rope_bwd(k64, up["k"], pos, freq, gamma=gk, **o)
    for L, t in ((Lg, dg64), (Lu, du64), (Lq, dq64.reshape(N, D)), (Lk, dk64.reshape(N, D))):
        d[L] = L.oracle(h64, t)
    rdx, rdgamma, _ = H.layernorm_bwd(x, sum(d[L]["dx"] for L in (Lg, Lu, Lq, Lk)), gamma)
    tol = 10 * TOL_F32
    assert O.rel_fro(host(qr), B.qk_rope(q64, pos, freq, gamma=gq, **o)) <= tol
    assert O.rel_fro(host(kr), B.qk_rope(k64, pos, freq, gamma=gk, **o)) <= tol
    assert O.rel_fro(host(y), d[Ld]["y"]) <= tol
    ref = [d[L][key] for L in layers for key in ("dq_R", "dq_P")] + [rdgamma, dgq64, dgk64]
    for got, want in zip([dx, *grads], [rdx, *ref]):
        assert O.rel_fro(host(got), want) <= tol
    n64 = B.grad_norm(ref)
    assert abs(float(norm) - n64) <= tol * n64
    # the clipped step on every triangle at once: the one tensor at a time on gradients clipped before
    hp = dict(step=2, lr=1e-3, weight_decay=0.01)
    tri = {"q": [t for L in layers for t in L.q], "dq": grads[:-3]}
    for s in "mv":
        tri[s] = [torch.full_like(t, 1e-4) for t in tri["q"]]
    alone = {s: [t.clone() for t in ts] for s, ts in tri.items()}
    P.poetx_adam_group(tri["q"], tri["dq"], tri["m"], tri["v"], norm=norm, max_norm=0.5 * n64, **hp)
    P.poetx_grad_clip(alone["dq"], norm, 0.5 * n64)
    for args in zip(*(alone[s] for s in ("q", "dq", "m", "v"))):
        P.poetx_adam_triu(*args, **hp)
    for s in ("q", "m", "v"):
        for one, other in zip(tri[s], alone[s]):
            assert torch.equal(one, other), s
    assert P.poetx_get_device_error() == 0


@pytest.mark.parametrize("kept", [True, False])
def test_norm_ffn_head_chain_fp32(P, kept):
    N, D, F, V = 150, 72, 136, 301
    r = np.random.default_rng(5)
    x = (r.standard_normal((N, D)) * 2).astype(np.float32)
    Wf = (r.standard_normal((2 * F, D)) / np.sqrt(D)).astype(np.float32)
    Wh = (r.standard_normal((V, F)) / np.sqrt(F)).astype(np.float32)
    t = r.integers(0, V, N).astype(np.int32)
    t[3] = -1
    up = np.full(N, 1 / (N - 1), np.float32)
    xd, Wfd, Whd = (dev(v, torch.float32) for v in (x, Wf, Wh))
    h, mean, rstd, a, z = _f32(N, D), _f32(N), _f32(N), _f32(N, F), _f32(N, 2 * F) if kept else None
    loss, da, dWh, dWf, dh, dx = _f32(N), _f32(N, F), _f32(V, F), _f32(2 * F, D), _f32(N, D), _f32(N, D)
    P.poetx_layernorm_fwd(xd, h, mean=mean, rstd=rstd)
    P.poetx_ffn_fwd(h, Wfd, a, z=z, act=P.GELU)
    P.poetx_head_ce(a, Whd, dev(t, torch.int32), loss, dloss=dev(up, torch.float32), dx=da, dW=dWh)
    P.poetx_ffn_bwd(h, Wfd, da, z=z, dx=dh, dW=dWf, act=P.GELU)
    P.poetx_layernorm_bwd(xd, dh, mean, rstd, dx)
    h64, _, _ = H.layernorm(x)
    a64, _ = B.ffn(h64, Wf, B.GELU)
    head = H.head_ce(a64, Wh, t, up)
    dh64, dWf64 = B.ffn_bwd(h64, Wf, head["dx"], B.GELU)
    rdx, _, _ = H.layernorm_bwd(x, dh64)
    for got, ref in ((a, a64), (loss, head["loss"]), (dWh, head["dW"]), (dWf, dWf64), (dx, rdx)):
        assert O.rel_fro(host(got), ref) <= 5 * TOL_F32
    assert P.poetx_get_device_error() == 0


def test_example_runs_and_its_gradients(P):
    """Finite losses; the slope of the fp32 loss along the triangles' gradient against a central
    difference over 2 x 0.02.  The loss near 8 is rounded to 2^-22 or so, which is 2e-5 of a slope of 1 over
    that distance; the difference's own error is the third derivative's share, some 0.02^2."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_block
    finally:
        sys.path.pop(0)
    losses, norms = train_block.train(steps=3, tokens=128, width=256, inner=512, vocab=503)
    assert np.isfinite(losses).all() and np.isfinite(norms).all() and min(norms) > 0
    slope, difference = train_block.check(tokens=256, width=256, inner=512, vocab=503)
    assert abs(slope - difference) <= 5e-3 * abs(difference), (slope, difference)
