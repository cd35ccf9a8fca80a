"""fp64 definitions of what stands between a transformer block's linears and behind their gradients:
the gated feed-forward block, the norms of queries and keys with the rotation by positions, the global
gradient norm and its clipping factor.

numpy, float64; matmul and fancy indexing are the only library primitives.  Test infrastructure
only: it shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

SILU, GELU = 0, 1


def activation(g, act):
    """(a(g), a'(g))."""
    g = np.asarray(g, np.float64)
    if act == SILU:
        e = np.exp(-np.abs(g))
        s = np.where(g >= 0, 1 / (1 + e), e / (1 + e))
        return g * s, s + g * s * (1 - s)
    c = np.sqrt(2 / np.pi)
    t = np.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), \
        0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g ** 2)


def glu(g, u, act):
    return activation(g, act)[0] * np.asarray(u, np.float64)


def glu_bwd(g, u, dh, act):
    a, d = activation(g, act)
    dh = np.asarray(dh, np.float64)
    return dh * u * d, dh * a


def ffn(x, W, act):
    """(h, z)."""
    z = np.asarray(x, np.float64) @ np.asarray(W, np.float64).T
    F = z.shape[1] // 2
    return glu(z[:, :F], z[:, F:], act), z


def ffn_bwd(x, W, dh, act, z=None):
    """(dx, dW), from the kept projections z or from new ones."""
    x, W = np.asarray(x, np.float64), np.asarray(W, np.float64)
    z = x @ W.T if z is None else np.asarray(z, np.float64)
    F = z.shape[1] // 2
    dz = np.concatenate(glu_bwd(z[:, :F], z[:, F:], dh, act), axis=1)
    return dz @ W, dz.T @ x


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


# 2^256 / (2 pi), rounded: a turn in integers.  (2 pi by Machin's formula, 320 bits.)
def _turn_bits(bits=256, more=64):
    one = 1 << (bits + more)

    def arctan_of_inverse(x):
        term = total = one // x
        k, sign = 1, -1
        while term:
            term //= x * x
            k += 2
            total += sign * (term // k)
            sign = -sign
        return total

    two_pi = 8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))  # times 2^(bits + more)
    return ((one << bits) + two_pi // 2) // two_pi


_TURN_BITS = 256
_INVERSE_TURN = _turn_bits(_TURN_BITS)


def _angles(pos, freq):
    """pos * freq (whole numbers by 64-bit numbers, both exact), modulo 2 pi where the product in 64 bits would
    have lost more than 2^-43 of a radian."""
    pos, freq = np.broadcast_arrays(pos, freq)
    angle = pos.astype(np.float64) * freq
    for i in zip(*np.nonzero(np.abs(angle) > 1024.0)):
        num, den = float(freq[i]).as_integer_ratio()  # den is a power of two
        scale = den << _TURN_BITS
        turns = (int(pos[i]) * num * _INVERSE_TURN) % scale
        if 2 * turns > scale:
            turns -= scale
        angle[i] = turns / scale * (2 * np.pi)
    return angle


def _rotate(x, pos, inv_freq, axis, interleaved, sign):
    """x [N, H, dh]; pos [axes, N]; the pairs turned by sign times their angles."""
    half = len(inv_freq)
    first, second = _pairs(2 * half, interleaved)
    ax = np.zeros(half, int) if axis is None else np.asarray(axis, int)
    angle = _angles(np.asarray(pos)[ax].T, np.asarray(inv_freq, np.float64))
    c, s = np.cos(angle)[:, None], sign * np.sin(angle)[:, None]
    y = x.copy()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., first] * s + x[..., second] * c
    return y


def qk_rope(x, pos, inv_freq, axis=None, interleaved=False, norm=True, gamma=None, eps=1e-6):
    n = np.asarray(x, np.float64)
    if norm:
        n = n / np.sqrt((n ** 2).mean(axis=-1, keepdims=True) + eps)
        if gamma is not None:
            n = n * gamma
    return _rotate(n, pos, inv_freq, axis, interleaved, 1.0)


def qk_rope_bwd(x, dy, pos, inv_freq, axis=None, interleaved=False, norm=True, gamma=None, eps=1e-6):
    """(dx, dgamma)."""
    dn = _rotate(np.asarray(dy, np.float64), pos, inv_freq, axis, interleaved, -1.0)
    if not norm:
        return dn, None
    x = np.asarray(x, np.float64)
    rstd = 1 / np.sqrt((x ** 2).mean(axis=-1, keepdims=True) + eps)
    h = x * rstd
    u = dn if gamma is None else dn * gamma
    return rstd * (u - h * (u * h).mean(axis=-1, keepdims=True)), (dn * h).sum(axis=(0, 1))


def grad_norm(grads):
    return np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))


def clip_factor(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6))
