"""Two sequence layers beside the nonlinear recurrence, each used three ways.

    python -m nonlinear_rnn_evaluation_amd.mixer

``Mixer`` mixes the recurrence with linear attention, on x [B, T, D]:

    h = diagonal GRU states of x                         pnr.evaluate       (parallel Newton)
    q, k, v, gate, a = slices of h W_in                  one projection
    o = linear attention, log decay = log sigmoid(a)     pnr.linear_attention
    y = group_norm(o by heads) * silu(gate)              pnr.group_norm
    out = y W_out

``prompt`` runs it over whole, possibly padded sequences and returns the states from which
``token`` continues, one token for each request, with the attention states in a pool;
``gradients`` runs it forward and back.  The projections are torch products; the rest runs in
the HIP library.

``StateSpace`` is a selective state space layer, on x [B, T, D]:

    x, z = halves of x W_in                              one projection
    u = silu(causal convolution of x)                    pnr.causal_conv
    dt, B, C = slices of u W_x, dt = dt W_dt
    y = selective scan of u, gated by silu(z)            pnr.selective_scan
    out = y W_out

with the same three methods.  Its ``gradients`` keeps the convolution's input, on request in 8 bits
(pnr.checkpoint_pack), and u not at all: u is made again from what was kept.
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


class StateSpace:
    """The layer's parameters: E channels of N states in G groups, W taps, step widths of rank R."""

    def __init__(self, D: int, E: int, N: int = 16, *, G: int = 1, W: int = 4, R: int = 8, seed: int = 0, device="cuda"):
        self.D, self.E, self.N, self.G, self.W, self.R = D, E, N, G, W, R
        g = torch.Generator().manual_seed(seed)
        self.sizes = [R, G * N, G * N]                                    # dt, B, C

        def draw(*shape, scale):
            return (torch.randn(*shape, generator=g) * scale).to(device)
        self.W_in = draw(D, 2 * E, scale=D ** -0.5)
        self.conv_w, self.conv_b = draw(E, W, scale=W ** -0.5), draw(E, scale=W ** -0.5)
        self.W_x = draw(E, sum(self.sizes), scale=E ** -0.5)
        self.W_dt = draw(R, E, scale=R ** -0.5)
        width = torch.exp(torch.rand(E, generator=g) * 4.6 - 6.9)         # step widths of 0.001 to 0.1
        self.dt_bias = (width + torch.log(-torch.expm1(-width))).to(device)
        self.A_log = torch.log(torch.arange(1.0, N + 1)).expand(E, N).contiguous().to(device)
        self.D_skip = torch.ones(E, device=device)
        self.W_out = draw(E, D, scale=E ** -0.5)

    def _inner(self, u):
        """What the scan takes besides u: dt, A, B, C; B and C are strided slices."""
        low, B, C = (u @ self.W_x).split(self.sizes, -1)
        shape = (self.G, self.N)
        return low, low @ self.W_dt, -torch.exp(self.A_log), B.unflatten(-1, shape), C.unflatten(-1, shape)

    def prompt(self, x, lens=None):
        """x [B, T, D], lens int32 [B]: dict(out [B, T, D], conv [B, W - 1, E] and S [B, E, N], the states after
        each row's last token).  What lies behind a row's end in x is not used, and in out not meaningful."""
        if lens is not None:
            live = torch.arange(x.shape[1], device=x.device)[None, :, None] < lens[:, None, None]
            x = torch.where(live, x, x.new_zeros(()))
        xs, z = (x @ self.W_in).chunk(2, -1)
        c = pnr.causal_conv(xs, self.conv_w, bias=self.conv_b, lens=lens)
        _, dt, A, B, C = self._inner(c["y"])
        r = pnr.selective_scan(c["y"], dt, A, B, C, D=self.D_skip, z=z, dt_bias=self.dt_bias, lens=lens)
        return dict(out=r["y"] @ self.W_out, conv=c["state"], S=r["state"])

    def token(self, x, conv, pool, slots):
        """x [B, D], one token for each request, whose states lie in slot slots[b] of the pools conv
        [n_slots, W - 1, E] and pool [n_slots, E, N], which are updated in place.  Returns out [B, D]."""
        xs, z = (x @ self.W_in).chunk(2, -1)
        u = pnr.causal_conv_step(xs, self.conv_w, conv, bias=self.conv_b, slots=slots)["y"]
        _, dt, A, B, C = self._inner(u)
        return pnr.selective_scan_step(u, dt, A, B, C, pool, D=self.D_skip, z=z, dt_bias=self.dt_bias, slots=slots)["y"] @ self.W_out

    def gradients(self, x, grad_out, keep=False):
        """out for x [B, T, D] and the gradients of <out, grad_out>: dict of x and of the parameters.  With keep,
        what the backward pass needs of the convolution's input waits in 8 bits: out is that of x, and the gradients
        are those at the rounded input, in everything that follows from it (u, dt, B and C)."""
        xs, z = (x @ self.W_in).chunk(2, -1)
        conv = dict(bias=self.conv_b)
        u = pnr.causal_conv(xs, self.conv_w, **conv)["y"]
        low, dt, A, B, C = self._inner(u)
        y = pnr.selective_scan(u, dt, A, B, C, D=self.D_skip, z=z, dt_bias=self.dt_bias)["y"]
        del u, low, dt, B, C
        out = y @ self.W_out
        kept = xs
        if keep:                                                          # xs and z are halves of one tensor: both go
            kept, z = pnr.checkpoint_pack(xs), z.contiguous()
        del xs
        # back: u again, the output projection, the scan, its inputs' projections, the convolution
        u = pnr.causal_conv(kept, self.conv_w, dtype=x.dtype, **conv)["y"]
        low, dt, A, B, C = self._inner(u)
        d = pnr.selective_scan_backward(u, dt, A, B, C, grad_out @ self.W_out.T, D=self.D_skip, z=z, dt_bias=self.dt_bias)
        grad_low = torch.cat([d["dt"] @ self.W_dt.T, d["B"].flatten(2), d["C"].flatten(2)], -1)
        dc = pnr.causal_conv_backward(kept, self.conv_w, d["u"] + grad_low @ self.W_x.T, **conv)
        grad_in = torch.cat([dc["x"], d["z"]], -1)

        def outer(a, b):
            return a.flatten(0, 1).T @ b.flatten(0, 1)
        return dict(out=out, x=grad_in @ self.W_in.T, W_in=outer(x, grad_in), conv_w=dc["weight"], conv_b=dc["bias"],
                    W_x=outer(u, grad_low), W_dt=outer(low, d["dt"]), dt_bias=d["dt_bias"], A_log=d["A"] * A,
                    D_skip=d["D"], W_out=outer(y, grad_out))


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
    layer = StateSpace(D=256, E=512)
    full, start = layer.prompt(x, lens), layer.prompt(x, short)
    conv, states, worst = torch.zeros(8, 3, 512, device="cuda"), torch.zeros(8, 512, 16, device="cuda"), 0.0
    conv[slots.long()], states[slots.long()] = start["conv"], start["S"]
    for i in range(10):
        at = short.long() + i
        out = layer.token(x[rows, at].contiguous(), conv, states, slots)
        worst = max(worst, (out - full["out"][rows, at]).abs().max().item())
    print(f"state space layer, prompt against token by token: largest difference {worst:.2e}")
    one = torch.ones_like(x)
    exact, kept = (layer.gradients(x, one, keep=k)["conv_w"] for k in (False, True))
    print(f"its taps' gradient from an input kept in 8 bits: off by {((kept - exact).norm() / exact.norm()).item():.1e} of its norm")
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
