"""Layer norm over many rows: every form that such calls take, with rings that turn several times,
against the definition in 64 bits.

Bounds per element: a bf16 result is rounded once, 2^-8 of it; statistics and fp32 arithmetic are held
to 1e-5 of the row's (or column's) scale, some 100 roundings."""
import pytest
import torch

from gpu_util import DEV, P, TOL_F32  # noqa: F401

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
N_ROWS = 6001  # 39 or 40 rows per SM, 19 or 20 per group of a pair
# 16-byte vectors of a row: a warp per row in its three sizes, the ring with one and with two vectors
# per thread, in one group and in two, at their limits
VECTORS = [7, 100, 128, 129, 200, 256, 257, 400, 512, 513, 777, 1024]


def _definition(x, dy, gamma, beta, eps, mean=None, rstd=None):
    x, dy, gamma, beta = x.double(), dy.double(), gamma.double(), beta.double()
    if mean is None:
        mean = x.mean(1)
        rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    mean, rstd = mean.double(), rstd.double()
    h = (x - mean[:, None]) * rstd[:, None]
    u = dy * gamma
    dx = rstd[:, None] * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True))
    return {"y": h * gamma + beta, "mean": mean, "rstd": rstd, "dx": dx, "dgamma": (dy * h).sum(0),
            "dbeta": dy.sum(0)}, h, u


def _run(P, x, dy, gamma, beta, eps=1e-5):
    N, D = x.shape
    o = {"y": torch.empty_like(x), "dx": torch.empty_like(x)}
    o["mean"], o["rstd"] = (torch.empty(N, device=DEV) for _ in range(2))
    o["dgamma"], o["dbeta"] = (torch.empty(D, device=DEV) for _ in range(2))
    P.poetx_layernorm_fwd(x, o["y"], gamma=gamma, beta=beta, mean=o["mean"], rstd=o["rstd"], eps=eps)
    P.poetx_layernorm_bwd(x, dy, o["mean"], o["rstd"], o["dx"], gamma=gamma, dgamma=o["dgamma"],
                          dbeta=o["dbeta"])
    torch.cuda.synchronize()
    assert P.poetx_get_device_error() == 0
    return o


def _inputs(N, D, dt, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x = (r(N, D) * (0.5 + r(N, 1).abs()) + r(N, 1)).to(DT[dt])
    return x, r(N, D).to(DT[dt]), 1 + 0.2 * r(D), r(D)


def _within(got, ref, u, scale, what):
    over = (got.double() - ref).abs() - (u * ref.abs() + TOL_F32 * scale)
    assert over.max().item() <= 0, (what, over.max().item(), over.argmax().item())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vectors", VECTORS)
def test_many_rows(P, vectors, dt):
    D = vectors * (8 if dt == "bf16" else 4)
    x, dy, gamma, beta = _inputs(N_ROWS, D, dt, vectors)
    got = _run(P, x, dy, gamma, beta)
    ref, h, u = _definition(x, dy, gamma, beta, 1e-5)
    half = 2.0 ** -8 if dt == "bf16" else 0.0
    row = lambda a: a.abs().amax(1, keepdim=True)
    _within(got["mean"], ref["mean"], 0, row(x.double())[:, 0], "mean")
    _within(got["rstd"], ref["rstd"], 0, ref["rstd"], "rstd")
    _within(got["y"], ref["y"], half, row(ref["y"]), "y")
    _within(got["dx"], ref["dx"], half, ref["rstd"][:, None] * row(u) * row(h), "dx")
    _within(got["dgamma"], ref["dgamma"], 0, (dy.double() * h).abs().sum(0), "dgamma")
    _within(got["dbeta"], ref["dbeta"], 0, dy.double().abs().sum(0), "dbeta")
    # the statistics are optional, the same bits without them
    y = torch.empty_like(x)
    P.poetx_layernorm_fwd(x, y, gamma=gamma, beta=beta)
    assert torch.equal(y, got["y"])


# few rows, and each form of many; widths whose reciprocal is not a power of two
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 4000])
@pytest.mark.parametrize("vectors", [100, 200, 500, 600])
def test_constant_rows_give_beta(P, vectors, N, dt):
    """A row of one value has no deviations, wherever it lies: y is beta, bit for bit."""
    D = vectors * (8 if dt == "bf16" else 4)
    _, dy, gamma, beta = _inputs(N, D, dt, vectors)
    value = 13.0 * 2.0 ** torch.arange(N, device=DEV).remainder(6)  # 13 to 416, exact in bf16
    x = value[:, None].expand(N, D).to(DT[dt]).contiguous()
    got = torch.empty_like(x)
    P.poetx_layernorm_fwd(x, got, gamma=gamma, beta=beta)
    assert torch.equal(got, beta.to(DT[dt]).expand(N, D))


@pytest.mark.parametrize("N", [3, 4000])
@pytest.mark.parametrize("vectors", [100, 200, 500, 1000])
def test_backward_far_from_zero(P, vectors, N):
    """Rows of 416 + N(0, 1) / 100 in fp32, with the forward's mean and rstd: x - mean is exact there,
    and the gradients keep it."""
    D = 4 * vectors
    x, dy, gamma, beta = _inputs(N, D, "f32", vectors)
    g = torch.Generator(device=DEV).manual_seed(9)
    x = 416 + torch.randn(N, D, generator=g, device=DEV) / 100
    got = _run(P, x, dy, gamma, beta)
    ref, h, u = _definition(x, dy, gamma, beta, 1e-5, got["mean"], got["rstd"])
    row = lambda a: a.abs().amax(1, keepdim=True)
    _within(got["dx"], ref["dx"], 0, ref["rstd"][:, None] * row(u), "dx")
    _within(got["dgamma"], ref["dgamma"], 0, (dy.double() * h).abs().sum(0), "dgamma")
    x.fill_(416.0)
    got = _run(P, x, dy, gamma, beta)
    assert (got["mean"] == 416).all() and not got["dgamma"].any()
