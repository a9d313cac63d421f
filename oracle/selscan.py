"""Selective scan, the causal convolution and 8-bit copies of activations, token by token (oracle;
test infrastructure only).

The definitions, in fp64.  Scan, for each row, channel e and state n (g the channel's group):
delta = softplus(dt + bias), h_t = exp(delta A) h_{t-1} + delta u B_t, y0 = C_t . h_t + D u,
y = y0 silu(z); gradients from the adjoint G_t = gy C_t + exp(delta_{t+1} A) G_{t+1} of the
states, gy = grad_y silu(z).  Convolution: y_t = act(b + sum_j w_j x_{t-W+1+j}).  Packing: 32
values on the least 2^e, e >= -126, of which the largest is at most 127.

Layouts follow the library: u, dt, z [B, T, E], B, C [B, T, G, N], A [E, N], states [B, E, N];
x [B, T, E], weight [E, W], states [B, W - 1, E]; lens [B].
"""
from __future__ import annotations

import numpy as np


def _softplus(x):
    return np.logaddexp(0.0, x)


def _sigmoid(x):
    return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


def _length(lens, b, T):
    return T if lens is None else int(np.clip(lens[b], 0, T))


def _widths(dt, bias, softplus):
    raw = dt if bias is None else dt + bias
    return (_softplus(raw), _sigmoid(raw)) if softplus else (raw, np.ones_like(raw))


def _walk(u, delta, A, Bc, h):
    """All states h_0..h_n of one row; Bc [n, E, N]."""
    hs = [h]
    for t in range(len(u)):
        hs.append(np.exp(delta[t][:, None] * A) * hs[-1] + (delta[t] * u[t])[:, None] * Bc[t])
    return np.stack(hs)


def selective_scan(u, dt, A, B, C, D=None, z=None, bias=None, softplus=True, state=None, lens=None):
    """(y [B, T, E], state [B, E, N]); zeros behind a row's end."""
    nb, T, E = u.shape
    rep = E // B.shape[2]
    y, out = np.zeros(u.shape), np.zeros((nb, E, A.shape[1]))
    delta, _ = _widths(dt, bias, softplus)
    for b in range(nb):
        n = _length(lens, b, T)
        Bc, Cc = np.repeat(B[b, :n], rep, 1), np.repeat(C[b, :n], rep, 1)
        hs = _walk(u[b, :n], delta[b, :n], A, Bc, np.zeros_like(out[b]) if state is None else state[b])
        y[b, :n] = (hs[1:] * Cc).sum(-1) + (0.0 if D is None else D * u[b, :n])
        if z is not None:
            y[b, :n] *= z[b, :n] * _sigmoid(z[b, :n])
        out[b] = hs[-1]
    return y, out


def selective_scan_grad(u, dt, A, B, C, gy, D=None, z=None, bias=None, softplus=True, state=None, lens=None,
                        gstate=None):
    """dict of the gradients of <y, gy> + <state, gstate> by name."""
    nb, T, E = u.shape
    G, N = B.shape[2:]
    rep = E // G
    g = {k: np.zeros(v.shape) for k, v in dict(u=u, dt=dt, A=A, B=B, C=C, z=u).items()}
    g["D"], g["dt_bias"], g["state"] = np.zeros(E), np.zeros(E), np.zeros((nb, E, N))
    delta, slope = _widths(dt, bias, softplus)
    for b in range(nb):
        n = _length(lens, b, T)
        Bc, Cc = np.repeat(B[b, :n], rep, 1), np.repeat(C[b, :n], rep, 1)
        hs = _walk(u[b, :n], delta[b, :n], A, Bc, np.zeros((E, N)) if state is None else state[b])
        adj = np.zeros((E, N)) if gstate is None else gstate[b].astype(np.float64)
        for t in range(n - 1, -1, -1):
            ut, d, gt = u[b, t], delta[b, t], gy[b, t].astype(np.float64)
            y0 = (hs[t + 1] * Cc[t]).sum(-1) + (0.0 if D is None else D * ut)
            if z is not None:
                s = _sigmoid(z[b, t])
                g["z"][b, t] = gt * y0 * s * (1 + z[b, t] * (1 - s))
                gt = gt * z[b, t] * s
            adj = adj + gt[:, None] * Cc[t]
            g["C"][b, t] = (gt[:, None] * hs[t + 1]).reshape(G, rep, N).sum(1)
            g["B"][b, t] = (adj * (d * ut)[:, None]).reshape(G, rep, N).sum(1)
            q = (adj * Bc[t]).sum(-1)
            g["u"][b, t] = d * q + (0.0 if D is None else D * gt)
            g["D"] += gt * ut
            adj = adj * np.exp(d[:, None] * A)
            gd = ut * q + (adj * hs[t] * A).sum(-1)
            g["A"] += adj * hs[t] * d[:, None]
            g["dt"][b, t] = gd * slope[b, t]
            g["dt_bias"] += g["dt"][b, t]
        g["state"][b] = adj
    return g


def _act(name, p):
    """act(p) and its derivative."""
    if name == "none":
        return p, np.ones_like(p)
    s = _sigmoid(p)
    return p * s, s * (1 + p * (1 - s))


def _inputs(x, state, W):
    return np.concatenate([np.zeros((W - 1, x.shape[1])) if state is None else state, x])


def causal_conv(x, weight, bias=None, act="silu", state=None, lens=None):
    """(y [B, T, E], state [B, W - 1, E])."""
    nb, T, E = x.shape
    W = weight.shape[1]
    y, out = np.zeros(x.shape), np.zeros((nb, W - 1, E))
    for b in range(nb):
        n = _length(lens, b, T)
        full = _inputs(x[b, :n], None if state is None else state[b], W)
        for t in range(n):
            y[b, t] = _act(act, (0.0 if bias is None else bias) + (full[t:t + W] * weight.T).sum(0))[0]
        out[b] = full[n:]
    return y, out


def causal_conv_grad(x, weight, gy, bias=None, act="silu", state=None, lens=None, gstate=None):
    nb, T, E = x.shape
    W = weight.shape[1]
    g = dict(x=np.zeros(x.shape), weight=np.zeros(weight.shape), bias=np.zeros(E), state=np.zeros((nb, W - 1, E)))
    for b in range(nb):
        n = _length(lens, b, T)
        full = _inputs(x[b, :n], None if state is None else state[b], W)
        gf = np.zeros(full.shape)
        if gstate is not None:
            gf[n:] += gstate[b]
        for t in range(n):
            p = (0.0 if bias is None else bias) + (full[t:t + W] * weight.T).sum(0)
            gp = gy[b, t] * _act(act, p)[1]
            gf[t:t + W] += gp * weight.T
            g["weight"] += (gp * full[t:t + W]).T
            g["bias"] += gp
        g["state"][b], g["x"][b, :n] = gf[:W - 1], gf[W - 1:]
    return g


def packed(x):
    """x [..., E] in 8 bits: (codes int8 [..., E], exponents uint8 [..., ceil(E / 32)], values)."""
    E = x.shape[-1]
    b = np.pad(x, [(0, 0)] * (x.ndim - 1) + [(0, -E % 32)]).reshape(*x.shape[:-1], (E + 31) // 32, 32)
    codes, exps = np.zeros(b.shape, np.int8), np.full(b.shape[:-1], 255, np.uint8)
    values = np.full(b.shape, np.nan)
    for i in np.ndindex(*b.shape[:-1]):
        most = np.abs(b[i]).max()
        if not np.isfinite(most):
            continue
        e = -126
        while most > 127.0 * 2.0 ** e:
            e += 1
        top = 63 if e == 122 else 127            # 64 * 2^122 is not an fp32 number
        codes[i], exps[i] = np.clip(np.rint(b[i] / 2.0 ** e), -top, top), e + 127
        values[i] = codes[i] * 2.0 ** e
    shape = (*x.shape[:-1], b.shape[-2] * 32)
    return codes.reshape(shape)[..., :E], exps, values.reshape(shape)[..., :E]
