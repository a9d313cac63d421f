"""Group norm with an activation, channels last, row by row (oracle; test infrastructure only).

n = (x - mean) / sqrt(var + eps) over a row's positions and a group's channels, z = n w + b,
y = act(z) or z act(gate); gradients by the chain rule, with the normalisation's Jacobian
dx = (u - mean(u) - n mean(u n)) / sqrt(var + eps), u = dz w.  fp64.
"""
from __future__ import annotations

import numpy as np

ACTS = ("none", "silu", "gelu")


def act(name, u):
    """act(u) and its derivative; gelu in its tanh form."""
    if name == "none":
        return u, np.ones_like(u)
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-u))
        return u * s, s * (1.0 + u * (1.0 - s))
    c = np.sqrt(2.0 / np.pi)
    th = np.tanh(c * (u + 0.044715 * u ** 3))
    return 0.5 * u * (1 + th), 0.5 * (1 + th) + 0.5 * u * (1 - th ** 2) * c * (1 + 3 * 0.044715 * u ** 2)


def _normed(x, groups, eps):
    """x [L, C]: normalised values, mean and 1 / sqrt(var + eps) per group."""
    L, C = x.shape
    xs = x.reshape(L, groups, C // groups)
    if L == 0:
        return x, np.zeros(groups), np.full(groups, 1.0 / np.sqrt(eps))
    mean = xs.mean((0, 2))
    r = 1.0 / np.sqrt(((xs - mean[:, None]) ** 2).mean((0, 2)) + eps)
    return ((xs - mean[:, None]) * r[:, None]).reshape(L, C), mean, r


def group_norm(x, groups, weight=None, bias=None, gate=None, activation="none", eps=1e-5, lens=None):
    """x [N, L, C]: (y, mean [N, groups], rstd [N, groups])."""
    N, L, C = x.shape
    y, mean, rstd = np.zeros(x.shape), np.zeros((N, groups)), np.zeros((N, groups))
    for i in range(N):
        n = L if lens is None else int(np.clip(lens[i], 0, L))
        z, mean[i], rstd[i] = _normed(x[i, :n], groups, eps)
        z = z if weight is None else z * weight + bias
        y[i, :n] = act(activation, z)[0] if gate is None else z * act(activation, gate[i, :n])[0]
    return y, mean, rstd


def group_norm_grad(gy, x, groups, weight=None, bias=None, gate=None, activation="none", eps=1e-5, lens=None):
    """dict of the gradients of <y, gy>: x, weight, bias, gate."""
    N, L, C = x.shape
    out = {"x": np.zeros(x.shape), "weight": np.zeros(C), "bias": np.zeros(C), "gate": np.zeros(x.shape)}
    w = np.ones(C) if weight is None else weight
    for i in range(N):
        n = L if lens is None else int(np.clip(lens[i], 0, L))
        if n == 0:
            continue
        h, _, r = _normed(x[i, :n], groups, eps)
        z = h if weight is None else h * w + bias
        if gate is None:
            dz = gy[i, :n] * act(activation, z)[1]
        else:
            a, da = act(activation, gate[i, :n])
            dz = gy[i, :n] * a
            out["gate"][i, :n] = gy[i, :n] * z * da
        out["weight"] += (dz * h).sum(0)
        out["bias"] += dz.sum(0)
        u, hs = (dz * w).reshape(n, groups, -1), h.reshape(n, groups, -1)
        m1, m2 = u.mean((0, 2), keepdims=True), (u * hs).mean((0, 2), keepdims=True)
        out["x"][i, :n] = (r[:, None] * (u - m1 - hs * m2)).reshape(n, C)
    return out
