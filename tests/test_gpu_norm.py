"""Layer norm forward and backward against the fp64 definition.

Tolerances, relative Frobenius error.  bf16 y and dx: one rounding of an fp32 result, 2^-9 of an
element at most (TOL_BF16_STEP).  fp32 outputs, mean and rstd: sums of at most 2^14 fp32 terms by
trees and partials, a few 2^-24 each (TOL_F32).  A mean is compared against the row's scale."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import DEV, P, TOL_BF16_STEP, TOL_F32, dev, host  # noqa: F401
from oracle import head_oracle as H

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# the 16-byte and the element forms of every register shape, the wide form, odd sizes, one element
SHAPES = [(1, 1), (5, 8), (3, 17), (1000, 104), (9, 1024), (33, 1027), (2, 2049), (700, 2000),
          (517, 4096), (31, 5001), (257, 8192), (6, 16384), (5, 20001)]


def _inputs(N, D, dt, seed):
    r = np.random.default_rng(seed)
    x = torch.tensor(r.standard_normal((N, D)) * 2 + 1.5).to(DT[dt])
    dy = torch.tensor(r.standard_normal((N, D))).to(DT[dt])
    gamma = (1 + 0.2 * r.standard_normal(D)).astype(np.float32)
    beta = r.standard_normal(D).astype(np.float32)
    return x, dy, gamma, beta


def _norms(P, x, dy, gamma, beta, eps=1e-5, acc=None):
    N, D = x.shape
    xd, dyd = x.to(DEV), dy.to(DEV)
    g = None if gamma is None else dev(gamma, torch.float32)
    b = None if beta is None else dev(beta, torch.float32)
    y, dx = torch.empty_like(xd), torch.empty_like(xd)
    mean, rstd = (torch.empty(N, device=DEV) for _ in range(2))
    dg, db = (torch.full((D,), float("nan") if acc is None else acc, device=DEV) for _ in range(2))
    P.poetx_layernorm_fwd(xd, y, gamma=g, beta=b, mean=mean, rstd=rstd, eps=eps)
    P.poetx_layernorm_bwd(xd, dyd, mean, rstd, dx, gamma=g, dgamma=dg, dbeta=db,
                          accumulate=acc is not None)
    torch.cuda.synchronize()
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dgamma": dg, "dbeta": db}


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,D", SHAPES)
@pytest.mark.parametrize("affine", [True, False], ids=["affine", "plain"])
def test_layernorm(P, N, D, dt, affine):
    x, dy, gamma, beta = _inputs(N, D, dt, 100 * N + D)
    if not affine:
        gamma = beta = None
    got = _norms(P, x, dy, gamma, beta)
    x64, dy64 = host(x), host(dy)
    y, mean, rstd = H.layernorm(x64, gamma, beta)
    dx, dgamma, dbeta = H.layernorm_bwd(x64, dy64, gamma)
    tol = TOL_BF16_STEP if dt == "bf16" else TOL_F32
    assert np.abs(host(got["mean"]) - mean).max() <= TOL_F32 * np.abs(x64).max()
    assert O.rel_fro(host(got["rstd"]), rstd) <= TOL_F32
    if D > 1:
        assert O.rel_fro(host(got["y"]), y) <= tol
        assert O.rel_fro(host(got["dgamma"]), dgamma) <= TOL_F32
        # at D = 8 or 17 dx is still of the size of its terms
        assert O.rel_fro(host(got["dx"]), dx) <= tol
    else:  # the row is its own mean
        assert np.abs(host(got["y"]) - y).max() <= tol * (1 if beta is None else np.abs(beta).max())
        assert not host(got["dx"]).any() and not host(got["dgamma"]).any()
    assert O.rel_fro(host(got["dbeta"]), dbeta) <= TOL_F32


def test_layernorm_parameter_gradients_accumulate_and_repeat(P):
    x, dy, gamma, beta = _inputs(300, 264, "bf16", 7)
    a, b = _norms(P, x, dy, gamma, beta), _norms(P, x, dy, gamma, beta)
    c = _norms(P, x, dy, gamma, beta, acc=0.5)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    for k in ("dgamma", "dbeta"):
        assert torch.equal(a[k] + 0.5, c[k]), k


def test_layernorm_constant_and_large_offset_rows(P):
    """A constant row has zero variance; a row far from zero keeps its deviations (the variance is
    taken around the mean: 1000 + N(0, 1) in fp32 holds them to 6e-5)."""
    x = torch.full((2, 4096), 3.0)
    x[1] = 1000 + torch.tensor(np.random.default_rng(0).standard_normal(4096), dtype=torch.float32)
    got = _norms(P, x, torch.ones_like(x), None, None)
    y, _, rstd = H.layernorm(host(x))
    assert not host(got["y"])[0].any()
    assert O.rel_fro(host(got["y"])[1], y[1]) <= 1e-4
    assert O.rel_fro(host(got["rstd"]), rstd) <= TOL_F32


def test_layernorm_nan_stays_in_its_row(P):
    x, dy, gamma, beta = _inputs(7, 520, "bf16", 8)
    x[3, 11] = float("nan")
    got = _norms(P, x, dy, gamma, beta)
    assert torch.isnan(got["y"][3]).all() and torch.isnan(got["dx"][3]).all()
    keep = [r for r in range(7) if r != 3]
    assert torch.isfinite(got["y"][keep]).all() and torch.isfinite(got["dx"][keep]).all()


def test_layernorm_optional_outputs_and_empty_batch(P):
    x, dy, gamma, beta = _inputs(40, 128, "f32", 9)
    full = _norms(P, x, dy, gamma, beta)
    xd, g = x.to(DEV), dev(gamma, torch.float32)
    y, dx, db = torch.empty_like(xd), torch.empty_like(xd), torch.empty(128, device=DEV)
    P.poetx_layernorm_fwd(xd, y, gamma=g, beta=dev(beta, torch.float32))
    assert torch.equal(y, full["y"])
    P.poetx_layernorm_bwd(xd, dy.to(DEV), full["mean"], full["rstd"], dx, gamma=g, dbeta=db)
    assert torch.equal(dx, full["dx"]) and torch.equal(db, full["dbeta"])
    dx.zero_()
    P.poetx_layernorm_bwd(xd, dy.to(DEV), full["mean"], full["rstd"], dx, gamma=g)
    assert torch.equal(dx, full["dx"])
    none, e = torch.empty(0, 128, device=DEV), torch.empty(0, device=DEV)
    P.poetx_layernorm_fwd(none, none.clone())
    P.poetx_layernorm_bwd(none, none.clone(), e, e, none.clone(), dbeta=db, accumulate=True)
    assert torch.equal(db, full["dbeta"])
    P.poetx_layernorm_bwd(none, none.clone(), e, e, none.clone(), dbeta=db)
    assert not db.any()


def test_layernorm_on_another_stream(P):
    x, dy, gamma, beta = _inputs(2000, 1024, "bf16", 10)
    ref = _norms(P, x, dy, gamma, beta)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    xd, dyd, g = x.to(DEV), dy.to(DEV), dev(gamma, torch.float32)
    dx, dg, db = torch.empty_like(xd), torch.empty(1024, device=DEV), torch.empty(1024, device=DEV)
    torch.cuda.synchronize()
    P.poetx_layernorm_bwd(xd, dyd, ref["mean"], ref["rstd"], dx, gamma=g, dgamma=dg, dbeta=db,
                          stream=s)
    s.synchronize()
    assert torch.equal(dx, ref["dx"]) and torch.equal(dg, ref["dgamma"])
    assert torch.equal(db, ref["dbeta"])


def test_layernorm_beyond_32_bit_offsets(P):
    """More than 2^31 elements: the last rows are the same as in a call of their own."""
    N, D = 264000, 8200
    free, _ = torch.cuda.mem_get_info()
    if free < 6 * N * D * 2:
        pytest.skip("needs 26 GB")
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.zeros(N, D, dtype=torch.bfloat16, device=DEV)
    dy = torch.zeros_like(x)
    tail = 40
    x[-tail:] = torch.randn(tail, D, generator=g, device=DEV).bfloat16()
    dy[-tail:] = torch.randn(tail, D, generator=g, device=DEV).bfloat16()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(N, device=DEV), torch.empty(N, device=DEV)
    dg, db = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    P.poetx_layernorm_fwd(x, y, mean=mean, rstd=rstd)
    P.poetx_layernorm_bwd(x, dy, mean, rstd, dx, dgamma=dg, dbeta=db)
    ref = _norms(P, x[-tail:].cpu(), dy[-tail:].cpu(), None, None)
    for got, k in ((y, "y"), (dx, "dx")):
        assert not got[:-tail].any()
        # (few and many rows take different forms: the same value up to its last rounding)
        assert O.rel_fro(host(got[-tail:]), host(ref[k])) <= 2.0 ** -8
    assert O.rel_fro(host(dg), host(ref["dgamma"])) <= TOL_F32
    assert O.rel_fro(host(db), host(ref["dbeta"])) <= TOL_F32
