"""Linear attention with a decay for each head, token by token (oracle; test infrastructure only).

The definition, in fp64: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, query heads
in consecutive groups sharing a state head; and its gradients, from the adjoint
D_t = scale q_t do_t^T + exp(g_{t+1}) D_{t+1} of the states:
dq_t = scale S_t do_t, dk_t = D_t v_t, dv_t = D_t^T k_t, dg_t = <D_t, exp(g_t) S_{t-1}>,
dS_0 = exp(g_1) D_1.  Every state is stored: small problems only.

Layouts follow the library: q [B, T, H, Dk], k [B, T, Hkv, Dk], v [B, T, Hkv, Dv],
g [Hkv] or [B, T, Hkv], states [B, Hkv, Dk, Dv], lens [B].
"""
from __future__ import annotations

import numpy as np


def _row(q, k, v, g, state, scale):
    """One batch row of its own length: outputs, all states S_0..S_n and the decays."""
    n, H, Dk = q.shape
    Hkv, Dv = v.shape[1:]
    qg = q.reshape(n, Hkv, H // Hkv, Dk)
    dec = np.exp(np.broadcast_to(g, (n, Hkv)))
    S = np.zeros((n + 1, Hkv, Dk, Dv))
    S[0] = 0.0 if state is None else state
    o = np.zeros((n, Hkv, H // Hkv, Dv))
    for t in range(n):
        S[t + 1] = dec[t][:, None, None] * S[t] + k[t][:, :, None] * v[t][:, None, :]
        o[t] = scale * (qg[t] @ S[t + 1])
    return o.reshape(n, H, Dv), S, dec


def linear_attention(q, k, v, g, scale, state=None, lens=None):
    """(o [B, T, H, Dv], state [B, Hkv, Dk, Dv]); zeros behind a row's end."""
    B, T, H, _ = q.shape
    o = np.zeros((B, T, H, v.shape[-1]))
    out = np.zeros((B, v.shape[2], k.shape[-1], v.shape[-1]))
    for b in range(B):
        n = T if lens is None else int(np.clip(lens[b], 0, T))
        o[b, :n], S, _ = _row(q[b, :n], k[b, :n], v[b, :n], g if g.ndim == 1 else g[b, :n],
                              None if state is None else state[b], scale)
        out[b] = S[-1]
    return o, out


def linear_attention_grad(q, k, v, g, scale, go, state=None, lens=None, gstate=None):
    """dict of the gradients of <o, go> + <state, gstate>: q, k, v, state, and log_decay as
    [B, T, Hkv] (``log_decay_head`` is its sum over rows and tokens)."""
    B, T, H, Dk = q.shape
    Hkv, Dv = v.shape[2:]
    G = H // Hkv
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dg, ds = np.zeros((B, T, Hkv)), np.zeros((B, Hkv, Dk, Dv))
    for b in range(B):
        n = T if lens is None else int(np.clip(lens[b], 0, T))
        _, S, dec = _row(q[b, :n], k[b, :n], v[b, :n], g if g.ndim == 1 else g[b, :n],
                         None if state is None else state[b], scale)
        D = np.zeros((Hkv, Dk, Dv)) if gstate is None else gstate[b].astype(np.float64)
        for t in range(n - 1, -1, -1):
            qt, dot = q[b, t].reshape(Hkv, G, Dk), go[b, t].reshape(Hkv, G, Dv)
            D = D + scale * np.swapaxes(qt, 1, 2) @ dot
            dq[b, t] = (scale * dot @ np.swapaxes(S[t + 1], 1, 2)).reshape(H, Dk)
            dk[b, t] = (D @ v[b, t][:, :, None])[..., 0]
            dv[b, t] = (k[b, t][:, None, :] @ D)[:, 0]
            D = dec[t][:, None, None] * D
            dg[b, t] = (D * S[t]).sum((1, 2))
        ds[b] = D
    return {"q": dq, "k": dk, "v": dv, "log_decay": dg, "log_decay_head": dg.sum((0, 1)), "state": ds}
