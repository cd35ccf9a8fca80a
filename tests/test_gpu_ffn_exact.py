"""The gated block's products element by element, the second bf16 piece of dz, added dW, and arrays of more
than 2^31 elements or vectors.

Tolerances.  R = 2^-8: a bf16 result's rounding.  A product of bf16 operands is off by C = 2^-14 of the sum of its
terms' magnitudes: the tensor core truncates when it adds 16 products into its accumulator, 2^-23 each, at most
512 adds between two hand-overs here.  dz is rounded to one piece (R) or two (R^2) before its products, and is off by
a few 2^-22 of its factors' magnitudes, which C covers.

Two pieces make dx and dW as exact as fp32 operands would: their error is then that of the result's rounding, 1.0
times it (the rest is some 2^-14 of terms against 2^-9).  Without the second piece it is 1.4 times, added twice or taken
from another row as much or more, so the bound of 1.15 tells them apart."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, P, host  # noqa: F401
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
R, C = 2.0 ** -8, 2.0 ** -14


def _inputs(N, D, F, seed, dt=BF):
    r = np.random.default_rng(seed)
    t = lambda s, *n: torch.tensor(r.standard_normal(n) * s).to(dt)
    return t(1, N, D), t(D ** -0.5, 2 * F, D), t(1.0 / N, N, F)


def _run(P, x, W, dh, act, kept, dW=None):
    N, D, F = x.shape[0], x.shape[1], W.shape[0] // 2
    xd, Wd = x.to(DEV), W.to(DEV)
    new = lambda *s: torch.full(s, float("nan"), dtype=x.dtype, device=DEV)
    h, z, dx = new(N, F), new(N, 2 * F), new(N, D)
    add = dW is not None
    dW = dW.to(DEV) if add else new(2 * F, D)
    P.poetx_ffn_fwd(xd, Wd, h, z=z, act=act)
    P.poetx_ffn_bwd(xd, Wd, dh.to(DEV), z=z if kept else None, dx=dx, dW=dW, act=act, accumulate=add)
    torch.cuda.synchronize()
    assert P.poetx_get_device_error() == 0
    return {k: host(t) for k, t in (("h", h), ("z", z), ("dx", dx), ("dW", dW))}


def _bounds(x, W, dh, act, z, pieces):
    """The definition's gradients, and how far products of dz may be off (without the result's rounding)."""
    F = z.shape[1] // 2
    dx, dW = B.ffn_bwd(x, W, dh, act, z)
    a = np.abs(B.activation(z[:, :F], act)[0])
    size = np.concatenate([1.2 * np.abs(dh * z[:, F:]), np.abs(dh) * a], 1)  # |a'| < 1.2
    off = R ** pieces + C
    return dx, dW, off * (size @ np.abs(W)), off * (size.T @ np.abs(x))


# few-row kernels of every token count, the 2-CTA products with dz in two pieces and in one; ends inside tiles
SHAPES = [(1, 264, 200), (2, 136, 328), (4, 520, 136), (7, 136, 72), (16, 264, 392), (17, 520, 264), (33, 72, 1000),
          (64, 264, 520), (65, 136, 264), (100, 520, 72), (128, 264, 1000), (129, 72, 136), (300, 264, 520),
          (513, 136, 264), (3, 16456, 16), (90, 16392, 24)]


@pytest.mark.parametrize("kept", [True, False], ids=["kept", "mem"])
@pytest.mark.parametrize("act", [B.SILU, B.GELU])
@pytest.mark.parametrize("N,D,F", SHAPES)
def test_every_element(P, N, D, F, act, kept):
    x, W, dh = _inputs(N, D, F, N + D + F)
    got = _run(P, x, W, dh, act, kept)
    x, W, dh = host(x), host(W), host(dh)
    h, z = B.ffn(x, W, act)
    dz = C * (np.abs(x) @ np.abs(W).T)
    assert (np.abs(got["z"] - z) <= R * np.abs(z) + dz).all()
    dh_off = 1.2 * np.abs(z[:, F:]) * dz[:, :F] + np.abs(z[:, :F]) * dz[:, F:]
    assert (np.abs(got["h"] - h) <= (R + C) * np.abs(h) + 1.1 * dh_off).all()
    # without the kept projections dz comes from the fp32 sums: their error is far below C of dz's factors
    dx, dW, dx_off, dW_off = _bounds(x, W, dh, act, got["z"] if kept else z, 2 if N <= 128 else 1)
    if not kept:  # dz moves with z: |d(dz)| <= |dh| (|a''| |u| + |a'|) of z's error
        move = np.abs(dh) * (1.2 * np.abs(z[:, F:]) * dz[:, :F] + 1.2 * dz[:, F:])
        move = np.concatenate([move, np.abs(dh) * 1.2 * dz[:, :F]], 1)
        dx_off, dW_off = dx_off + move @ np.abs(W), dW_off + move.T @ np.abs(x)
    assert (np.abs(got["dx"] - dx) <= R * np.abs(dx) + dx_off).all()
    assert (np.abs(got["dW"] - dW) <= R * np.abs(dW) + dW_off).all()


def _times_rounding(got, ref):
    """The error, in errors of the rounded exact result."""
    rounded = host(torch.tensor(ref).to(BF))
    return np.linalg.norm(got - ref) / np.linalg.norm(rounded - ref)


@pytest.mark.parametrize("kept", [True, False], ids=["kept", "mem"])
@pytest.mark.parametrize("N,D,F", [
    # dz from the elementwise kernel (kept; mem beyond the few-row kernel's width), from the CUDA cores (one row, up
    # to four of small blocks) and from the few-row products; its pieces to the kernel of up to 16, 32 and 64 rows
    # and to the 2-CTA products
    (1, 2056, 1000), (2, 520, 520), (3, 2056, 264), (4, 264, 1416), (5, 1032, 2056), (16, 520, 1000), (17, 264, 2056),
    (32, 1032, 520), (33, 520, 264), (64, 264, 1000), (65, 520, 1000), (100, 1032, 520), (128, 264, 2056),
    (12, 16456, 40), (100, 16456, 24)])
def test_second_piece_of_dz(P, N, D, F, kept):
    x, W, dh = _inputs(N, D, F, 3 * N + D + F)
    got = _run(P, x, W, dh, B.SILU, kept)
    x, W, dh = host(x), host(W), host(dh)
    dx, dW = B.ffn_bwd(x, W, dh, B.SILU, got["z"] if kept else None)
    if not kept and D > 16384:  # by way of z in bf16
        dx, dW = B.ffn_bwd(x, W, dh, B.SILU, got["z"])
    assert _times_rounding(got["dx"], dx) <= 1.15
    assert _times_rounding(got["dW"], dW) <= 1.15


@pytest.mark.parametrize("N,D,F", [(200, 520, 1000), (1000, 264, 520)])
def test_one_piece_above_128_rows(P, N, D, F):
    """The rounding of dz beside the result's own, of the same size: the root of two times it."""
    x, W, dh = _inputs(N, D, F, 5 * N)
    got = _run(P, x, W, dh, B.SILU, True)
    dx, dW = B.ffn_bwd(host(x), host(W), host(dh), B.SILU, got["z"])
    assert _times_rounding(got["dx"], dx) <= 1.5
    assert _times_rounding(got["dW"], dW) <= 1.5


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,F", [(8, 8), (136, 72), (264, 1000), (1032, 264), (2056, 40)])
@pytest.mark.parametrize("N", [1, 6, 13, 20, 50, 100, 200])
def test_added_dW(P, N, D, F, dt):
    x, W, dh = _inputs(N, D, F, N + D + F, BF if dt == "bf16" else torch.float32)
    base = torch.tensor(np.random.default_rng(1).standard_normal((2 * F, D))).to(x.dtype)
    got = _run(P, x, W, dh, B.SILU, True, base)
    x, W, dh, base = host(x), host(W), host(dh), host(base)
    if dt == "f32":
        # fp32: dz and its products to some 2^-20 of the terms, the sum rounded once more
        dx, dW, dx_off, dW_off = _bounds(x, W, dh, B.SILU, got["z"], 1)
        r, off = 2.0 ** -23, 2.0 ** -18 / (R + C)
    else:
        dx, dW, dx_off, dW_off = _bounds(x, W, dh, B.SILU, got["z"], 2 if N <= 128 else 1)
        r, off = R, 1.0
    assert (np.abs(got["dx"] - dx) <= r * np.abs(dx) + off * dx_off).all()
    assert (np.abs(got["dW"] - (dW + base)) <= r * np.abs(dW + base) + 2.0 ** -22 * np.abs(base) + off * dW_off).all()


@pytest.fixture
def room():
    """Skips a test that the GPU has too little memory for; gives back afterwards what it took."""
    def needs(gigabytes):
        torch.cuda.empty_cache()
        if torch.cuda.mem_get_info()[0] < gigabytes << 30:
            pytest.skip(f"needs {gigabytes} GB")
    yield needs
    torch.cuda.empty_cache()


def _rows_of(N, some):
    """A [N] mask of the rows that hold something."""
    m = torch.zeros(N, dtype=torch.bool, device=DEV)
    m[some] = True
    return m


@pytest.mark.parametrize("halves", [True, False], ids=["halves", "two_launches"])
def test_glu_beyond_32_bits(P, room, halves):
    """More than 2^31 elements with rows apart from each other; more than 2^31 vectors, which take two launches
    (8191 rows in the first)."""
    F = 1 << 21
    N, some = (600, [0, 300, 511, 512, 599]) if halves else (8250, [0, 1023, 1024, 4096, 8190, 8191, 8192, 8249])
    room(20 if halves else 115)
    g = torch.Generator(device=DEV).manual_seed(2)
    if halves:
        z = torch.zeros(N, 2 * F, dtype=BF, device=DEV)
        gate, up = z[:, :F], z[:, F:]
    else:
        gate, up = (torch.zeros(N, F, dtype=BF, device=DEV) for _ in range(2))
    dh = torch.zeros(N, F, dtype=BF, device=DEV)
    for r in some:
        for t in (gate, up, dh):
            t[r] = torch.randn(F, generator=g, device=DEV).to(BF)
    small = [t[some].contiguous() for t in (gate, up, dh)]
    want = [torch.empty_like(small[0]) for _ in range(3)]
    P.poetx_glu_fwd(small[0], small[1], want[0])
    P.poetx_glu_bwd(*small, want[1], want[2])
    torch.cuda.synchronize()
    # the few rows by themselves are right (the first and the last of them) ...
    for i in (0, -1):
        v = [host(t[i]) for t in small]
        ref = [B.glu(v[0], v[1], B.SILU), *B.glu_bwd(*v, B.SILU)]
        for w, r in zip(want, ref):
            assert (np.abs(host(w[i]) - r) <= R * np.abs(r) + 1e-5 * (np.abs(r) + 1e-2 * np.abs(r).max())).all()
    # ... and the same among all rows; the others give zeros
    others = ~_rows_of(N, some)

    def same(t, w):
        assert torch.equal(t[some], w)
        for i in range(0, N, 64):
            assert not t[i:i + 64][others[i:i + 64]].any()

    h = torch.full((N, F), float("nan"), dtype=BF, device=DEV)
    P.poetx_glu_fwd(gate, up, h)
    same(h, want[0])
    del h
    P.poetx_glu_bwd(gate, up, dh, gate, up)  # in place
    same(gate, want[1])
    same(up, want[2])


def test_ffn_with_projections_beyond_32_bits(P, room):
    """z and dz of more than 2^31 elements, through the products of many rows."""
    N, D, F = 600, 8, 1 << 21
    room(40)
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(N, D, generator=g, device=DEV).to(BF)
    W = (torch.randn(2 * F, D, generator=g, device=DEV) / 3).to(BF)
    dh = (torch.randn(N, F, generator=g, device=DEV) / 64).to(BF)
    new = lambda *s: torch.full(s, float("nan"), dtype=BF, device=DEV)
    h, z = new(N, F), new(N, 2 * F)
    P.poetx_ffn_fwd(x, W, h, z=z)
    some = [0, 255, 256, 511, 512, 599]
    ref = x[some].double() @ W.double().t()
    off = C * (x[some].double().abs() @ W.double().abs().t())
    assert ((z[some].double() - ref).abs() <= R * ref.abs() + off).all()
    rh = torch.nn.functional.silu(ref[:, :F]) * ref[:, F:]
    h_off = 1.2 * ref[:, F:].abs() * off[:, :F] + ref[:, :F].abs() * off[:, F:]
    assert ((h[some].double() - rh).abs() <= (R + C) * rh.abs() + 1.1 * h_off).all()
    del ref, off, rh, h_off
    for kept in (True, False):
        dx, dW = new(N, D), new(2 * F, D)
        P.poetx_ffn_bwd(x, W, dh, z=z if kept else None, dx=dx, dW=dW)
        torch.cuda.synchronize()
        assert P.poetx_get_device_error() == 0
        # a token's dx, and the first and the last features' dW
        zz = z[some].double() if kept else x[some].double() @ W.double().t()
        s = torch.sigmoid(zz[:, :F])
        a, d = zz[:, :F] * s, s + zz[:, :F] * s * (1 - s)
        dz = torch.cat([dh[some].double() * zz[:, F:] * d, dh[some].double() * a], 1)
        # (dz's rounding: errors of either sign over four million terms, R of each at most; a bound of
        # six of their deviations)
        off = 6 * R * (dz ** 2 @ W.double() ** 2).sqrt() + C * (dz.abs() @ W.double().abs())
        rdx = dz @ W.double()
        assert ((dx[some].double() - rdx).abs() <= R * rdx.abs() + off).all()
        for f in (0, F - 1):
            zf = (z[:, [f, F + f]] if kept else x.double() @ W[[f, F + f]].double().t()).double()
            s = torch.sigmoid(zf[:, 0])
            d = dh[:, f].double()
            dg, du = d * zf[:, 1] * (s + zf[:, 0] * s * (1 - s)), d * zf[:, 0] * s
            for row, v in ((f, dg), (F + f, du)):
                r = v @ x.double()
                off = (R + C) * 1.2 * ((v.abs() + 1e-3 * d.abs()) @ x.double().abs())
                assert ((dW[row].double() - r).abs() <= R * r.abs() + off).all()
