"""The gated product and the gated feed-forward block against the fp64 definitions.

Tolerances.  A bf16 rounding is off by at most half a step, 2^-8 of the value.  Elementwise bf16
results: one rounding of fp32 arithmetic (a few 2^-22).  Products, relative Frobenius error: h and z
carry one rounding; dx and dW the rounding of dz and their own, in a mean over the terms no more than
two roundings.  fp32: sums of six products of bf16 pieces, TOL_F32."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import DEV, P, TOL_F32, dev, host  # noqa: F401
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
R = 2.0 ** -8  # one bf16 rounding
EXTRA = 1e-4   # fp32 sums of products, against it


def _glu_inputs(N, F, dt, seed):
    r = np.random.default_rng(seed)
    return [torch.tensor(r.standard_normal((N, F)) * s).to(DT[dt]) for s in (3.0, 1.0, 1.0)]


def _near(got, ref, dt):
    """Elementwise: one rounding and the arithmetic before it; a derivative near its zero is as
    exact as its terms."""
    scale = np.abs(ref) + 1e-2 * (np.abs(ref).max() if ref.size else 0)
    tol = R * np.abs(ref) + 1e-5 * scale if dt == "bf16" else 2e-6 * scale
    return (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", [B.SILU, B.GELU])
@pytest.mark.parametrize("N,F", [(1, 8), (3, 8), (7, 24), (130, 264), (33, 13824), (1000, 1096)])
@pytest.mark.parametrize("halves", [False, True])
def test_glu(P, N, F, act, dt, halves):
    g, u, dh = _glu_inputs(N, F, dt, N + F + act)
    ref, (rdg, rdu) = B.glu(host(g), host(u), act), B.glu_bwd(host(g), host(u), host(dh), act)
    if halves:  # of one array, and the gradients of another
        z = torch.cat([g, u], 1).to(DEV)
        gd, ud = z[:, :F], z[:, F:]
        dz = torch.empty_like(z)
        dg, du = dz[:, :F], dz[:, F:]
    else:
        gd, ud = g.to(DEV), u.to(DEV)
        dg, du = torch.empty_like(gd), torch.empty_like(ud)
    h = torch.empty(N, F, dtype=DT[dt], device=DEV)
    P.poetx_glu_fwd(gd, ud, h, act=act)
    P.poetx_glu_bwd(gd, ud, dh.to(DEV), dg, du, act=act)
    torch.cuda.synchronize()
    assert _near(host(h), ref, dt)
    assert _near(host(dg), rdg, dt) and _near(host(du), rdu, dt)
    P.poetx_glu_bwd(gd, ud, dh.to(DEV), gd, ud, act=act)  # in place
    assert torch.equal(gd, dg) and torch.equal(ud, du)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", [B.SILU, B.GELU])
def test_glu_far_gates(P, act, dt):
    """Gates far from zero: 0 or g itself, no NaN; an infinite gate of the positive side and NaN."""
    inf = float("inf")
    g = torch.tensor([[200.0, -200.0, 1e30, -1e30, inf, float("nan"), 0.0, -20.0]]).to(DT[dt])
    u = torch.full((1, 8), 2.0).to(DT[dt])
    h = torch.empty(1, 8, dtype=DT[dt], device=DEV)
    P.poetx_glu_fwd(g.to(DEV), u.to(DEV), h, act=act)
    got = host(h)[0]
    assert got[0] == 2 * host(g)[0, 0] and got[2] == 2 * host(g)[0, 2] and got[4] == inf
    assert got[1] == 0 and got[3] == 0 and got[6] == 0 and np.isnan(got[5])
    ref = B.glu(host(g)[:, 7:], [[2.0]], act)[0, 0]
    # in fp64 the tanh form has lost this tail, so only SiLU's is compared
    assert act == B.GELU and abs(got[7]) < 1e-9 or abs(got[7] - ref) <= 1.1 * R * abs(ref)


def _ffn_inputs(N, D, F, dt, seed):
    r = np.random.default_rng(seed)
    x = torch.tensor(r.standard_normal((N, D))).to(DT[dt])
    W = torch.tensor(r.standard_normal((2 * F, D)) / np.sqrt(D)).to(DT[dt])
    dh = torch.tensor(r.standard_normal((N, F)) / max(N, 1)).to(DT[dt])
    return x, W, dh


def _run(P, x, W, dh, act, kept, dx=True, dW=True, keep_z=True, **kw):
    N, D, F = x.shape[0], x.shape[1], W.shape[0] // 2
    xd, Wd, dhd = x.to(DEV), W.to(DEV), dh.to(DEV)
    new = lambda *s: torch.full(s, float("nan"), dtype=x.dtype, device=DEV)
    h, z = new(N, F), new(N, 2 * F) if keep_z else None
    P.poetx_ffn_fwd(xd, Wd, h, z=z, act=act)
    out = {"h": h, "z": z, "dx": new(N, D) if dx else None, "dW": new(2 * F, D) if dW else None}
    P.poetx_ffn_bwd(xd, Wd, dhd, z=z if kept else None, dx=out["dx"], dW=out["dW"], act=act, **kw)
    torch.cuda.synchronize()
    assert P.poetx_get_device_error() == 0
    return out


SHAPES = [(1, 8, 8), (2, 64, 128), (5, 72, 40), (16, 256, 1000), (17, 264, 2056), (40, 192, 136),
          (65, 128, 4096), (128, 520, 808), (129, 64, 64), (256, 136, 520), (300, 512, 1416),
          (257, 1032, 264), (1021, 328, 648),
          # beyond the few-row kernel's width; more features than SMs times 128; several accumulators' K
          (3, 16456, 16), (2, 64, 20000), (70, 72, 20008), (200, 4168, 136)]


@pytest.mark.parametrize("kept", [True, False], ids=["kept", "mem"])
@pytest.mark.parametrize("act", [B.SILU, B.GELU])
@pytest.mark.parametrize("N,D,F", SHAPES)
def test_ffn_bf16(P, N, D, F, act, kept):
    x, W, dh = _ffn_inputs(N, D, F, "bf16", 7 * N + D + F)
    got = _run(P, x, W, dh, act, kept)
    h, z = B.ffn(host(x), host(W), act)
    assert O.rel_fro(host(got["z"]), z) <= R + EXTRA
    assert O.rel_fro(host(got["h"]), h) <= R + EXTRA
    # the gradients of the kept projections as they are, or of the inputs
    dx, dW = B.ffn_bwd(host(x), host(W), host(dh), act, host(got["z"]) if kept else None)
    tol = 2 * R + EXTRA
    assert O.rel_fro(host(got["dx"]), dx) <= tol
    assert O.rel_fro(host(got["dW"]), dW) <= tol


@pytest.mark.parametrize("kept", [True, False], ids=["kept", "mem"])
@pytest.mark.parametrize("N,D,F", [(1, 8, 8), (5, 72, 40), (130, 264, 392), (300, 512, 1000)])
@pytest.mark.parametrize("act", [B.SILU, B.GELU])
def test_ffn_f32(P, N, D, F, act, kept):
    x, W, dh = _ffn_inputs(N, D, F, "f32", 5 * N + D + F)
    got = _run(P, x, W, dh, act, kept)
    h, z = B.ffn(host(x), host(W), act)
    dx, dW = B.ffn_bwd(host(x), host(W), host(dh), act)
    assert O.rel_fro(host(got["z"]), z) <= TOL_F32
    for k, ref in (("h", h), ("dx", dx), ("dW", dW)):  # the product behind another: twice
        assert O.rel_fro(host(got[k]), ref) <= 2 * TOL_F32, k


@pytest.mark.parametrize("N,dt", [(40, "bf16"), (200, "bf16"), (70, "f32")])
def test_ffn_options(P, N, dt):
    """The same bits whatever else is asked for; dW added to what is there."""
    x, W, dh = _ffn_inputs(N, 136, 328, dt, N)
    full = _run(P, x, W, dh, B.SILU, True)
    again = _run(P, x, W, dh, B.SILU, True)
    for k in full:
        assert torch.equal(full[k], again[k]), k
    h = torch.empty_like(full["h"])
    P.poetx_ffn_fwd(x.to(DEV), W.to(DEV), h)
    assert torch.equal(h, full["h"])
    only = _run(P, x, W, dh, B.SILU, True, dW=False)
    assert torch.equal(only["dx"], full["dx"])
    only = _run(P, x, W, dh, B.SILU, True, dx=False)
    assert torch.equal(only["dW"], full["dW"])
    base = torch.randn(full["dW"].shape, generator=torch.Generator().manual_seed(1)).to(DT[dt])
    dW = base.to(DEV)
    P.poetx_ffn_bwd(x.to(DEV), W.to(DEV), dh.to(DEV), z=full["z"], dW=dW, accumulate=True)
    ref = B.ffn_bwd(host(x), host(W), host(dh), B.SILU, host(full["z"]))[1] + host(base)
    assert O.rel_fro(host(dW), ref) <= (2 * R if dt == "bf16" else TOL_F32)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ffn_rows_on_their_own(P, dt):
    """Each row's result is its own: a NaN row leaves the others' bits alone."""
    for N in (33, 200):
        x, W, dh = _ffn_inputs(N, 72, 200, dt, 3)
        ref = _run(P, x, W, dh, B.SILU, True, dW=False)
        x[7, 3] = float("nan")
        got = _run(P, x, W, dh, B.SILU, True, dW=False)
        keep = [i for i in range(N) if i != 7]
        for k in ("h", "z", "dx"):
            assert torch.isnan(got[k][7]).all(), k
            assert torch.equal(got[k][keep], ref[k][keep]), k


@pytest.mark.parametrize("N,dt", [(40, "bf16"), (200, "bf16"), (40, "f32"), (200, "f32")])
def test_ffn_infinite_upstream(P, N, dt):
    """An infinite upstream gradient makes dz infinite in its feature: dx there is infinite or NaN as IEEE sums
    are, dW's two rows infinite (one row of x meets it), and no other row of dx or dW sees it."""
    x, W, dh = _ffn_inputs(N, 72, 64, dt, 11)
    ref = _run(P, x, W, dh, B.SILU, True)
    dh[5, 9] = float("inf")
    got = _run(P, x, W, dh, B.SILU, True)
    keep = [i for i in range(N) if i != 5]
    rows = [i for i in range(128) if i not in (9, 73)]
    assert torch.equal(got["dx"][keep], ref["dx"][keep]) and torch.equal(got["dW"][rows], ref["dW"][rows])
    z = host(got["z"])
    dz = B.glu_bwd(z[:, :64], z[:, 64:], host(dh), B.SILU)
    with np.errstate(invalid="ignore"):
        dx = dz[0][5, 9] * host(W)[9] + dz[1][5, 9] * host(W)[73]
        dW = [d[5, 9] * host(x)[5] for d in dz]
    assert np.array_equal(host(got["dx"][5]), dx, equal_nan=True)
    for r, w in zip((9, 73), dW):
        assert np.array_equal(host(got["dW"][r]), w, equal_nan=True)


def test_ffn_empty_batch(P):
    W = torch.randn(48, 64, device=DEV).bfloat16()
    x, h = torch.empty(0, 64, device=DEV).bfloat16(), torch.empty(0, 24, device=DEV).bfloat16()
    dW = torch.ones(48, 64, device=DEV).bfloat16()
    P.poetx_ffn_fwd(x, W, h)
    P.poetx_ffn_bwd(x, W, h.clone(), dW=dW, accumulate=True)
    assert (dW == 1).all()
    P.poetx_ffn_bwd(x, W, h.clone(), dW=dW)
    assert not dW.any()
    P.poetx_glu_fwd(h, h, h.clone())
    P.poetx_glu_bwd(h, h, h, h.clone(), h.clone())


@pytest.mark.parametrize("N", [1, 20, 150])
def test_ffn_writes_only_its_rows(P, N):
    x, W, dh = _ffn_inputs(N, 72, 136, "bf16", N)
    xd, Wd, dhd = x.to(DEV), W.to(DEV), dh.to(DEV)
    big = {k: torch.full((N + 3, w), 7.0, dtype=torch.bfloat16, device=DEV)
           for k, w in (("h", 136), ("z", 272), ("dx", 72))}
    P.poetx_ffn_fwd(xd, Wd, big["h"][:N], z=big["z"][:N])
    P.poetx_ffn_bwd(xd, Wd, dhd, z=big["z"][:N], dx=big["dx"][:N])
    torch.cuda.synchronize()
    for k, t in big.items():
        assert (t[N:] == 7).all(), k


def test_ffn_on_another_stream_and_in_a_graph(P):
    x, W, dh = _ffn_inputs(140, 128, 264, "bf16", 5)
    ref = _run(P, x, W, dh, B.SILU, False)
    xd, Wd, dhd = x.to(DEV), W.to(DEV), dh.to(DEV)
    h, dx, dW = (torch.zeros_like(ref[k]) for k in ("h", "dx", "dW"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    P.poetx_ffn_fwd(xd, Wd, h, stream=s)
    P.poetx_ffn_bwd(xd, Wd, dhd, dx=dx, dW=dW, stream=s)
    s.synchronize()
    assert torch.equal(h, ref["h"]) and torch.equal(dx, ref["dx"]) and torch.equal(dW, ref["dW"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.poetx_ffn_fwd(xd, Wd, h)
        P.poetx_ffn_bwd(xd, Wd, dhd, dx=dx, dW=dW)
    for t in (h, dx, dW):
        t.zero_()
    xd.copy_(xd.roll(1, 0)), dhd.copy_(dhd.roll(1, 0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, ref["h"].roll(1, 0)) and torch.equal(dx, ref["dx"].roll(1, 0))
    assert O.rel_fro(host(dW), host(ref["dW"])) <= 2 * R  # (other order of its sums)


@pytest.mark.parametrize("kept", [True, False], ids=["kept", "mem"])
@pytest.mark.parametrize("act", [B.SILU, B.GELU])
@pytest.mark.parametrize("N,D,F", [
    (1, 136, 808), (2, 264, 72), (3, 8, 4096), (4, 520, 200), (7, 1032, 24), (8, 128, 1000), (9, 136, 520),
    (16, 2056, 328), (17, 72, 136), (32, 264, 392), (33, 264, 392),
    # several blocks of tokens, the last of one token or seven
    (64, 136, 72), (65, 1032, 40), (199, 264, 520), (512, 64, 64), (97, 1600, 8),
    # more column tiles than places on the GPU; few rows of W to a warp
    (3, 40968, 16), (16, 20488, 8)])
def test_ffn_f32_few_rows(P, N, D, F, act, kept):
    x, W, dh = _ffn_inputs(N, D, F, "f32", 3 * N + D + F)
    got = _run(P, x, W, dh, act, kept)
    h, z = B.ffn(host(x), host(W), act)
    dx, dW = B.ffn_bwd(host(x), host(W), host(dh), act)
    assert O.rel_fro(host(got["z"]), z) <= TOL_F32
    for k, ref in (("h", h), ("dx", dx), ("dW", dW)):
        assert O.rel_fro(host(got[k]), ref) <= 2 * TOL_F32, k


@pytest.mark.parametrize("kept", [True, False], ids=["kept", "mem"])
@pytest.mark.parametrize("N,D,F", [(1, 264, 4096), (1, 8, 8), (1, 16456, 24), (1, 4104, 4104), (2, 1032, 808),
                                   (2, 4104, 4104), (3, 136, 72), (4, 2056, 520), (4, 72, 1000), (6, 4104, 72),
                                   (8, 2056, 520), (9, 264, 200),
                                   (3, 40968, 16), (8, 8, 20000), (7, 2056, 8200),
                                   # units of 128 rows and columns: one of both, ends inside them, more
                                   # blocks of columns than SMs, several jobs of a CTA
                                   (64, 8, 8), (9, 128, 64), (16, 136, 72), (33, 1032, 4104), (12, 20488, 72),
                                   (32, 72, 30008), (64, 2056, 1000), (20, 4104, 1416), (65, 264, 200)])
def test_ffn_bf16_few_rows(P, N, D, F, kept):
    x, W, dh = _ffn_inputs(N, D, F, "bf16", 11 * N + D + F)
    got = _run(P, x, W, dh, B.GELU, kept)
    h, z = B.ffn(host(x), host(W), B.GELU)
    assert O.rel_fro(host(got["z"]), z) <= R + EXTRA and O.rel_fro(host(got["h"]), h) <= R + EXTRA
    dx, dW = B.ffn_bwd(host(x), host(W), host(dh), B.GELU, host(got["z"]) if kept else None)
    for k, ref in (("dx", dx), ("dW", dW)):
        assert O.rel_fro(host(got[k]), ref) <= 2 * R + EXTRA, k


@pytest.mark.parametrize("N,dt", [(1, "bf16"), (8, "bf16"), (11, "bf16"), (64, "bf16"), (2, "f32"),
                                  (8, "f32"), (15, "f32"), (25, "f32")])
def test_ffn_options_few_rows(P, N, dt):
    test_ffn_options(P, N, dt)


@pytest.mark.parametrize("N,dt", [(7, "bf16"), (15, "bf16"), (50, "bf16"), (8, "f32"), (14, "f32"),
                                  (30, "f32")])
def test_ffn_few_rows_on_their_own(P, N, dt):
    """A NaN row of x and an infinite upstream gradient stay in their rows."""
    x, W, dh = _ffn_inputs(N, 136, 264, dt, 23)
    ref = _run(P, x, W, dh, B.SILU, False)
    x[N - 1, 3] = float("nan")
    got = _run(P, x, W, dh, B.SILU, False)
    for k in ("h", "z", "dx"):
        assert torch.isnan(got[k][N - 1]).all(), k
        assert torch.equal(got[k][:N - 1], ref[k][:N - 1]), k
    x, W, dh = _ffn_inputs(N, 136, 264, dt, 23)
    dh[0, 9] = float("inf")
    got = _run(P, x, W, dh, B.SILU, False)
    rows = [i for i in range(528) if i not in (9, 273)]
    assert torch.equal(got["dx"][1:], ref["dx"][1:]) and torch.equal(got["dW"][rows], ref["dW"][rows])
    assert not torch.isfinite(got["dx"][0]).any() and not torch.isfinite(got["dW"][[9, 273]]).any()


@pytest.mark.parametrize("N,dt", [(5, "bf16"), (21, "bf16"), (5, "f32")])
def test_ffn_few_rows_leave_what_lies_behind(P, N, dt):
    """Outputs inside larger arrays: nothing before or behind them is written, and the workspace ends
    where its size says."""
    D, F = 72, 136
    x, W, dh = (t.to(DEV) for t in _ffn_inputs(N, D, F, dt, 4))
    T = DT[dt]
    pad = 64

    def room(*shape):
        n = int(np.prod(shape))
        flat = torch.full((n + 2 * pad,), 7.0, dtype=T, device=DEV)
        return flat, flat[pad:pad + n].view(*shape)

    fh, h = room(N, F)
    fz, z = room(N, 2 * F)
    fx, dx = room(N, D)
    fw, dW = room(2 * F, D)
    P.poetx_ffn_fwd(x, W, h, z=z)
    for zz in (z, None):
        n = P.poetx_ffn_bwd_workspace_bytes(P.F32 if dt == "f32" else P.BF16, N, D, F, zz is not None)
        ws = torch.full((n + 256,), 0x5a, dtype=torch.uint8, device=DEV)
        P.poetx_ffn_bwd(x, W, dh, z=zz, dx=dx, dW=dW, ws=ws[:n])
        torch.cuda.synchronize()
        assert (ws[n:] == 0x5a).all()
    for flat in (fh, fz, fx, fw):
        assert (flat[:pad] == 7).all() and (flat[-pad:] == 7).all()


@pytest.mark.parametrize("N,dt", [(3, "f32"), (20, "f32"), (2, "bf16"), (40, "bf16")])
def test_ffn_few_rows_at_once_and_captured(P, N, dt):
    """Two streams at the same time, then two graphs that share a workspace, replayed after each other with
    other inputs."""
    x, W, dh = _ffn_inputs(N, 264, 1000, dt, N)
    ref = _run(P, x, W, dh, B.SILU, False)
    xd, Wd, dhd = x.to(DEV), W.to(DEV), dh.to(DEV)
    outs = [[torch.zeros_like(ref[k]) for k in ("h", "dx", "dW")] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (h, dx, dW) in zip(streams, outs):
            P.poetx_ffn_fwd(xd, Wd, h, stream=s)
            P.poetx_ffn_bwd(xd, Wd, dhd, dx=dx, dW=dW, stream=s)
    torch.cuda.synchronize()
    for out in outs:
        for k, t in zip(("h", "dx", "dW"), out):
            assert torch.equal(t, ref[k]), k
    code = P.F32 if dt == "f32" else P.BF16
    n = max(P.poetx_ffn_fwd_workspace_bytes(code, N, 264, 1000),
            P.poetx_ffn_bwd_workspace_bytes(code, N, 264, 1000, False))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    ins = [(xd.clone(), dhd.clone()) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, (xi, di), (h, dx, dW) in zip(graphs, ins, outs):
        with torch.cuda.graph(g):
            P.poetx_ffn_fwd(xi, Wd, h, ws=ws)
            P.poetx_ffn_bwd(xi, Wd, di, dx=dx, dW=dW, ws=ws)
    ins[1][0].copy_(xd * 2), ins[1][1].copy_(dhd * 0.5)
    other = _run(P, x * 2, W, dh * 0.5, B.SILU, False)
    for _ in range(2):
        for t in outs[0] + outs[1]:
            t.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for want, out in ((ref, outs[0]), (other, outs[1])):
            for k, t in zip(("h", "dx", "dW"), out):
                assert torch.equal(t, want[k]), k


@pytest.mark.parametrize("N,dt", [(2, "f32"), (11, "f32"), (5, "bf16")])
def test_ffn_few_rows_beyond_32_bits(P, N, dt):
    """W and dW of more than 2^31 elements: the last rows are read, multiplied and written where they are."""
    D, F, K = 16384, 70000, 8
    T = DT[dt]
    g = torch.Generator().manual_seed(N)
    W = torch.zeros(2 * F, D, dtype=T, device=DEV)
    last = [(torch.randn(K, D, generator=g) / 128).to(T) for _ in range(2)]
    W[F - K:F], W[2 * F - K:] = last[0].to(DEV), last[1].to(DEV)
    x = torch.randn(N, D, generator=g).to(T)
    dh = torch.zeros(N, F, dtype=T)
    dh[:, F - K:] = torch.randn(N, K, generator=g).to(T)
    new = lambda *s: torch.full(s, float("nan"), dtype=T, device=DEV)
    h, dx, dW = new(N, F), new(N, D), new(2 * F, D)
    P.poetx_ffn_fwd(x.to(DEV), W, h)
    P.poetx_ffn_bwd(x.to(DEV), W, dh.to(DEV), dx=dx, dW=dW)
    torch.cuda.synchronize()
    assert P.poetx_get_device_error() == 0
    small = np.concatenate([host(last[0]), host(last[1])])
    rh, _ = B.ffn(host(x), small, B.SILU)
    rdx, rdW = B.ffn_bwd(host(x), small, host(dh[:, F - K:]), B.SILU)
    tol = 2 * R + EXTRA if dt == "bf16" else 2 * TOL_F32
    assert not h[:, :F - K].any() and O.rel_fro(host(h[:, F - K:]), rh) <= tol
    assert O.rel_fro(host(dx), rdx) <= tol
    got = np.concatenate([host(dW[F - K:F]), host(dW[2 * F - K:])])
    assert O.rel_fro(got, rdW) <= tol
    dW[F - K:F].zero_(), dW[2 * F - K:].zero_()
    assert not dW.any()
