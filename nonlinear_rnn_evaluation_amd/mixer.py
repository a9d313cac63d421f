"""A sequence layer that mixes a nonlinear recurrence with linear attention, used three ways.

    python -m nonlinear_rnn_evaluation_amd.mixer

One layer, on x [B, T, D]:

    h = diagonal GRU states of x                         pnr.evaluate       (parallel Newton)
    q, k, v, gate, a = slices of h W_in                  one projection
    o = linear attention, log decay = log sigmoid(a)     pnr.linear_attention
    y = group_norm(o by heads) * silu(gate)              pnr.group_norm
    out = y W_out

``prompt`` runs it over whole, possibly padded sequences and returns the states from which
``token`` continues, one token for each request, with the attention states in a pool;
``gradients`` runs it forward and back.  The projections are torch products; the rest runs in
the HIP library.
"""
from __future__ import annotations

import torch

from . import pnr


class Mixer:
    """The layer's parameters: H query heads of size Dk and Dv on H_kv state heads."""

    def __init__(self, D: int, H: int, H_kv: int, Dk: int, Dv: int, *, seed: int = 0, device="cuda"):
        self.D, self.H, self.H_kv, self.Dk, self.Dv = D, H, H_kv, Dk, Dv
        g = torch.Generator().manual_seed(seed)
        self.sizes = [H * Dk, H_kv * Dk, H_kv * Dv, H * Dv, H_kv]        # q, k, v, gate, a

        def draw(*shape, scale):
            return (torch.randn(*shape, generator=g) * scale).to(device)
        self.W = draw(3 * D, D, scale=D ** -0.5)                          # GRU: input weights, gates r, z, n
        self.U = draw(3, D, scale=0.5)                                    # ... elementwise recurrent weights
        self.W_in = draw(D, sum(self.sizes), scale=D ** -0.5)
        self.W_out = draw(H * Dv, D, scale=(H * Dv) ** -0.5)
        self.norm_w, self.norm_b = torch.ones(H * Dv, device=device), torch.zeros(H * Dv, device=device)

    def _states(self, x, h0):
        r = pnr.evaluate(pnr.CELL_GRU_DIAG, self.W, self.U, x, h0=h0, max_iters=64, tol=1e-6)
        if r["status"] != pnr.OK:
            raise pnr.PnrError(f"the recurrence did not converge (status {r['status']})")
        return r["h"]

    def _project(self, h):
        """q, k, v, gate as strided slices of one projection, and the log decay."""
        q, k, v, gate, a = (h @ self.W_in).split(self.sizes, -1)
        return (q.unflatten(-1, (self.H, self.Dk)), k.unflatten(-1, (self.H_kv, self.Dk)),
                v.unflatten(-1, (self.H_kv, self.Dv)), gate.contiguous(), torch.nn.functional.logsigmoid(a + 3.0))

    def _normed(self, o, gate):
        """The gated norm by heads: every token is a row of its own."""
        C = self.H * self.Dv
        return pnr.group_norm(o.reshape(-1, 1, C), self.H, weight=self.norm_w, bias=self.norm_b,
                              gate=gate.reshape(-1, 1, C), act=pnr.ACT_SILU)

    def prompt(self, x, lens=None):
        """x [B, T, D], lens int32 [B] (row b has min(max(lens[b], 0), T) tokens): dict(out [B, T, D],
        h [B, D] and S, the states after each row's last token; a row without one hands the initial states
        on, zeros).  What lies behind a row's end in x is not read, and in out not meaningful."""
        n = torch.full((x.shape[0],), x.shape[1], device=x.device) if lens is None else lens.long().clamp(0, x.shape[1])
        if lens is not None:        # the recurrence runs over whole rows: zeros converge and stay finite
            x = torch.where(torch.arange(x.shape[1], device=x.device)[None, :, None] < n[:, None, None], x, x.new_zeros(()))
        h = self._states(x, None)
        q, k, v, gate, g = self._project(h)
        r = pnr.linear_attention(q, k, v, g, lens=lens)
        y = self._normed(r["o"], gate)["y"].view(*x.shape[:2], -1)
        last = h[torch.arange(len(h), device=h.device), (n - 1).clamp(min=0)]
        return dict(out=y @ self.W_out, S=r["state"], h=torch.where(n[:, None] > 0, last, torch.zeros_like(last)))

    def token(self, x, h, pool, slots):
        """x [B, D], one token for each request: h [B, D] its GRU state, its attention state in slot
        slots[b] of the pool, which is updated in place.  Returns (out [B, D], h)."""
        h = self._states(x[:, None], h)[:, 0].contiguous()
        q, k, v, gate, g = self._project(h)
        o = pnr.linear_attention_step(q, k, v, g, pool, slots=slots)["o"]
        return self._normed(o, gate)["y"].view(len(x), -1) @ self.W_out, h

    def gradients(self, x, grad_out):
        """out for x [B, T, D] and the gradients of <out, grad_out>: dict of x and of the parameters."""
        B, T, _ = x.shape
        h = self._states(x, None)
        q, k, v, gate, g = self._project(h)
        att = pnr.linear_attention(q, k, v, g)
        n = self._normed(att["o"], gate)
        y = n["y"].view(B, T, -1)
        # back: the output projection, the gated norm, the attention, the input projection, the recurrence
        grad_y = (grad_out @ self.W_out.T).reshape(n["y"].shape)
        C = n["y"].shape[-1]
        dn = pnr.group_norm_backward(grad_y, att["o"].reshape(-1, 1, C), self.H, n["mean"], n["rstd"],
                                     weight=self.norm_w, bias=self.norm_b, gate=gate.reshape(-1, 1, C), act=pnr.ACT_SILU)
        da = pnr.linear_attention_backward(q, k, v, g, dn["x"].view(B, T, self.H, self.Dv))
        grad_a = da["log_decay"] * (1 - g.exp())                          # through log sigmoid
        grad_p = torch.cat([da["q"].flatten(2), da["k"].flatten(2), da["v"].flatten(2),
                            dn["gate"].view(B, T, -1), grad_a], -1)
        grad_h = grad_p @ self.W_in.T
        dr = pnr.backward(pnr.CELL_GRU_DIAG, self.W, self.U, x, h, grad_h, want=("x", "W", "U"))
        return dict(out=y @ self.W_out, x=dr["x"], W=dr["W"], U=dr["U"], norm_w=dn["weight"], norm_b=dn["bias"],
                    W_in=h.flatten(0, 1).T @ grad_p.flatten(0, 1), W_out=y.flatten(0, 1).T @ grad_out.flatten(0, 1))


def main():
    m = Mixer(D=256, H=8, H_kv=4, Dk=64, Dv=64)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(3, 200, 256, generator=gen, device="cuda")
    lens = torch.tensor([200, 150, 17], dtype=torch.int32, device="cuda")
    whole = m.prompt(x, lens)
    # the same sequences, the last tokens of each decoded one at a time from a shorter prompt
    short = (lens - 10).to(torch.int32)
    part = m.prompt(x, short)
    pool = torch.zeros(8, 4, 64, 64, device="cuda")
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    pool[slots.long()] = part["S"]
    h, rows, worst = part["h"].contiguous(), torch.arange(3, device="cuda"), 0.0
    for i in range(10):
        at = short.long() + i
        out, h = m.token(x[rows, at].contiguous(), h, pool, slots)
        worst = max(worst, (out - whole["out"][rows, at]).abs().max().item())
    print(f"prompt against token by token: largest difference {worst:.2e}")
    target = torch.randn(x.shape, generator=gen, device="cuda")
    loss = []
    for _ in range(5):
        out = m.gradients(x, torch.zeros_like(x))["out"]
        g = m.gradients(x, 2 * (out - target) / out.numel())
        loss.append(((out - target) ** 2).mean().item())
        for name in ("W", "U", "W_in", "W_out", "norm_w", "norm_b"):
            getattr(m, name).sub_(200.0 * g[name])
    print("training loss:", " ".join(f"{v:.4f}" for v in loss))


if __name__ == "__main__":
    main()
