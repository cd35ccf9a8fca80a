"""Infinities and NaN in the linear head's inputs: what the definition calls NaN is NaN, it stays in
the rows (and vocabulary entries) it belongs to, and a logit of -inf is a probability of 0."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, P, dev, host  # noqa: F401
from oracle import head_oracle as H
from test_gpu_head import _ce, _distill, _inputs, _near

pytestmark = pytest.mark.gpu

# bf16: the product of few rows and the one of many; fp32: one for both
ROWS = [("bf16", 40), ("bf16", 140), ("f32", 40)]


@pytest.mark.parametrize("dt,N", ROWS)
@pytest.mark.parametrize("T", [1.0, 2.0])
def test_distill_teacher_logits_not_finite(P, dt, N, T):
    """A NaN or +inf among a row's present entries leaves the row no distribution: its loss and its
    dx are NaN, and dW where the row's entries are.  Absent entries are not read."""
    V = 900
    x, W, _, g = _inputs(N, V, 64, dt, 30)
    r = np.random.default_rng(2)
    idx = np.stack([r.permutation(V)[:6] for _ in range(N)]).astype(np.int32)
    u = r.uniform(-3, 6, (N, 6)).astype(np.float32)
    u[2, 3] = np.nan
    u[5, 0] = np.inf
    u[6] = np.nan
    u[7] = np.inf
    u[8], u[8, 2] = -np.inf, np.nan
    idx[9, 1:], u[9, 0] = -1, np.nan
    bad = [2, 5, 6, 7, 8, 9]
    idx[10, 2], u[10, 2] = -1, np.nan
    idx[11, 2], u[11, 2] = -1, np.inf
    u[12, 4] = -np.inf
    ok = np.setdiff1d(np.arange(N), bad)
    for grads in (False, True):
        got = _distill(P, x, W, idx, u, g, T, grads=grads)
        assert np.isnan(host(got["loss"])[bad]).all()
        ref = H.head_distill(host(x)[ok], host(W), idx[ok], u[ok], g[ok] if grads else None, T)
        ref["lse"] = H.head_distill(host(x), host(W), idx, u, None, T)["lse"]
        for k in ("loss", "dx"):
            if k in got:
                got[k] = got[k][torch.as_tensor(ok, device=DEV)]
        _near({k: v for k, v in got.items() if k != "dW"}, ref, dt)
    got = _distill(P, x, W, idx, u, g, T)
    assert np.isnan(host(got["dx"])[bad]).all()
    named = np.unique(idx[bad][idx[bad] >= 0])
    dW = host(got["dW"])
    assert np.isnan(dW[idx[[2, 5, 6, 7]].ravel()]).all()
    g0 = g.copy()
    full = H.head_distill(host(x), host(W), idx, np.where(np.isfinite(u) | (u < 0), u, 0), g0, T)
    rest = np.setdiff1d(np.arange(V), named)  # there p alone counts
    _near({"dW": torch.as_tensor(dW[rest])}, {"dW": full["dW"][rest]}, dt)


@pytest.mark.parametrize("dt,N", ROWS)
@pytest.mark.parametrize("how", ["nan", "inf-inf"])
def test_target_logit_not_a_number(P, dt, N, how):
    """A vocabulary entry whose logit is NaN takes every row with it, those that have it as their
    target too; an ignored row's loss is 0 all the same."""
    x, W, t, g = _inputs(N, 700, 64, dt, 31)
    if how == "nan":
        W[300] = float("nan")
    else:
        x[:, :2] = x[:, :2].abs() + 0.1
        W[300, 0], W[300, 1] = float("inf"), float("-inf")
    t[3], t[4], t[5] = 300, -1, 300
    kept = t >= 0
    for grads in (False, True):
        got = _ce(P, x, W, t, g, dx=grads, dW=grads)
        assert np.isnan(host(got["lse"])).all()
        assert np.isnan(host(got["loss"])[kept]).all() and host(got["loss"])[4] == 0
    assert np.isnan(host(got["dx"])[kept]).all()
    idx = t[:, None].astype(np.int32)
    got = _distill(P, x, W, idx, np.zeros((N, 1), np.float32), g)
    assert np.isnan(host(got["loss"])[kept]).all() and np.isnan(host(got["dx"])[kept]).all()


@pytest.mark.parametrize("N", [40, 300])
@pytest.mark.parametrize("where", ["row", "element"])
def test_fp32_infinite_weights(P, N, where):
    """fp32: an entry whose logit is -inf has probability 0, with fp32 accuracy for all others."""
    x, W, t, g = _inputs(N, 700, 64, "f32", 32)
    x = x.abs() + 0.1 if where == "row" else x
    x[:, 5] = x[:, 5].abs() + 0.1
    out = np.zeros(700, bool)
    out[128:256] = out[300] = True
    W[torch.as_tensor(out), 0 if where == "row" else 5:(64 if where == "row" else 6)] = float("-inf")
    t[out[t]] = 5
    keep, place = ~out, np.cumsum(~out) - 1
    ref = H.head_ce(host(x), host(W)[keep], place[t], g)
    got = _ce(P, x, W, t, g)
    assert not host(got["dW"])[out].any()  # p is 0
    got["dW"] = got["dW"][torch.as_tensor(keep, device=DEV)]
    del got["dx"]  # 0 x -inf
    _near(got, ref, "f32")


def test_fp32_infinities_give_what_the_definition_gives(P):
    """+inf in W, and infinities and NaN in x: NaN where the log-sum-exp of such logits is NaN."""
    x, W, t, g = _inputs(60, 500, 64, "f32", 33)
    x[:, 5] = x[:, 5].abs() + 0.1
    W[10, 5] = float("inf")
    got = _ce(P, x, W, t, g, dx=False, dW=False)
    assert np.isnan(host(got["lse"])).all() and np.isnan(host(got["loss"])).all()
    x, W, t, g = _inputs(60, 500, 64, "f32", 34)
    x[7, 3], x[8, 9], x[9, 11] = float("inf"), float("-inf"), float("nan")
    got = _ce(P, x, W, t, g, dW=False)
    ok = np.setdiff1d(np.arange(60), [7, 8, 9])
    for k in ("loss", "lse", "dx"):
        assert np.isnan(host(got[k])[[7, 8, 9]]).all(), k
        got[k] = got[k][torch.as_tensor(ok, device=DEV)]
    ref = H.head_ce(host(x)[ok], host(W), t[ok], g[ok])
    _near(got, ref, "f32")


def test_fp32_largest_numbers(P):
    """Values that bf16 rounds to infinity are finite in fp32: a logit of 8 from the largest one."""
    x, W, t, g = _inputs(50, 500, 64, "f32", 35)
    W[:, 1] = 0
    x[:, 1] = 2.0 ** -125
    W[50, 1], W[51, 1] = torch.finfo(torch.float32).max, -3.4e38
    t[:5] = 50
    ref = H.head_ce(host(x), host(W), t, g)
    got = _ce(P, x, W, t, g, dx=False)  # (dx reaches the size of W)
    _near(got, ref, "f32")
