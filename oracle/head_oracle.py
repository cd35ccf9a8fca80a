"""fp64 definitions of the training head's operators: layer norm, the linear head's softmax cross
entropy and distillation from a teacher's top logits, with their gradients.

numpy, float64; matmul and fancy indexing are the only library primitives.  Test infrastructure
only: it shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def layernorm(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd) of the rows of x."""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mean, rstd


def layernorm_bwd(x, dy, gamma=None, eps=1e-5):
    """(dx, dgamma, dbeta) for the upstream gradient dy."""
    h, _, rstd = layernorm(x, None, None, eps)
    dy = np.asarray(dy, np.float64)
    u = dy if gamma is None else dy * gamma
    dx = rstd[:, None] * (u - u.mean(axis=1, keepdims=True) -
                          h * (u * h).mean(axis=1, keepdims=True))
    return dx, (dy * h).sum(axis=0), dy.sum(axis=0)


def _logsumexp(z):
    top = z.max(axis=1)
    return top + np.log(np.exp(z - top[:, None]).sum(axis=1))


def head_ce(x, W, target, dloss=None, z_loss=0.0):
    """dict of loss, lse and, with dloss, dx and dW; rows with target < 0 are ignored."""
    x, W = np.asarray(x, np.float64), np.asarray(W, np.float64)
    z = x @ W.T
    lse = _logsumexp(z)
    rows = np.nonzero(target >= 0)[0]
    loss = np.zeros(x.shape[0])
    loss[rows] = lse[rows] - z[rows, target[rows]] + z_loss * lse[rows] ** 2
    out = {"loss": loss, "lse": lse}
    if dloss is not None:
        dz = np.zeros_like(z)
        dz[rows] = np.exp(z[rows] - lse[rows, None]) * (1 + 2 * z_loss * lse[rows])[:, None]
        dz[rows, target[rows]] -= 1.0
        dz *= np.asarray(dloss, np.float64)[:, None]
        out["dx"], out["dW"] = dz @ W, dz.T @ x
    return out


def head_distill(x, W, t_index, t_logit, dloss=None, temperature=1.0):
    """dict of loss = T^2 KL(teacher || student), lse and, with dloss, dx and dW; entries with a
    negative index are absent, rows without entries (or with all of them -inf) are ignored; a NaN or
    +inf among a row's entries leaves it no distribution: NaN."""
    T = float(temperature)
    x, W = np.asarray(x, np.float64), np.asarray(W, np.float64)
    z = x @ W.T / T
    lse = _logsumexp(z)
    loss = np.zeros(x.shape[0])
    dz = np.zeros_like(z)
    for r in range(x.shape[0]):
        ks = [k for k in range(t_index.shape[1])
              if t_index[r, k] >= 0 and t_logit[r, k] != -np.inf]
        if not ks:
            continue
        u = np.asarray(t_logit[r, ks], np.float64) / T
        logq = u - (u.max() + np.log(np.exp(u - u.max()).sum()))
        logp = z[r] - lse[r]
        dz[r] = np.exp(logp)
        for k, lq in zip(ks, logq):
            loss[r] += T * T * np.exp(lq) * (lq - logp[t_index[r, k]])
            dz[r, t_index[r, k]] -= np.exp(lq)
    out = {"loss": loss, "lse": lse}
    if dloss is not None:
        dz *= np.asarray(dloss, np.float64)[:, None] * T
        out["dx"], out["dW"] = dz @ W, dz.T @ x
    return out
