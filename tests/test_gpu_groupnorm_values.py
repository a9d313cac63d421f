"""Group norm on values far from the ordinary: finite inputs give the formula's values.

Tolerance: relative 2^-8 for each bf16 element (its own rounding, twice), and 2^-17 of each fp32 element, as
the hardware exponential and reciprocal (2^-22 each) in a few steps of fp32 allow."""
import numpy as np
import pytest
import torch

import oracle as O
from nonlinear_rnn_evaluation_amd import pnr

GATES = [0.0, 1.0, -1.0, 5.0, -5.0, 9.0, -9.0, 30.0, -30.0, 1e4, -1e4, 2e13, -2e13, 3e19, -3e19, 1e38, -1e38]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("L", [1, 6])
def test_gates_of_any_finite_size(L, act, dtype):
    """An activation's value and its derivative over the whole range: the derivative of a large gate is 1 or 0."""
    C = 24
    gen = torch.Generator().manual_seed(3)
    gate = torch.tensor([GATES[i % len(GATES)] for i in range(4 * L * C)]).reshape(4, L, C).to(dtype).cuda()
    x = torch.randn(4, L, C, generator=gen).to(dtype).cuda()
    # small enough that no product with a gate of 1e38 leaves the range
    gy = (torch.randn(4, L, C, generator=gen) * 1e-3).to(dtype).cuda()
    a = {"silu": pnr.ACT_SILU, "gelu": pnr.ACT_GELU}[act]
    f = pnr.group_norm(x, 3, gate=gate, act=a)
    d = pnr.group_norm_backward(gy, x, 3, f["mean"], f["rstd"], gate=gate, act=a)
    X, G, Y = (t.double().cpu().numpy() for t in (x, gate, gy))
    want = O.group_norm_grad(Y, X, 3, gate=G, activation=act)["gate"]
    got = d["gate"].double().cpu().numpy()
    assert np.isfinite(got).all()
    tol = 2.0 ** (-8 if dtype == torch.bfloat16 else -17)
    # the normalised x under the gate is good to 2^-17 of its size, about 1; products below 1e-30 may be flushed
    assert (np.abs(got - want) <= tol * np.abs(want) + 2.0 ** -17 * np.abs(Y) + 1e-30).all()
    y, ref = f["y"].double().cpu().numpy(), O.group_norm(X, 3, gate=G, activation=act)[0]
    assert (np.abs(y - ref) <= tol * np.abs(ref) + 2.0 ** -17 * np.abs(np.where(G > 0, G, 1.0)) + 1e-30).all()


@pytest.mark.gpu
@pytest.mark.parametrize("L", [1, 5])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_rows_without_positions_have_zero_gradients_whatever_the_weights(bad, gated, L):
    gen = torch.Generator().manual_seed(4)
    x, gy, gate = (torch.randn(6, L, 16, generator=gen).cuda() for _ in range(3))
    w, b = torch.ones(16, device="cuda"), torch.zeros(16, device="cuda")
    w[3], b[9] = bad, bad
    lens = torch.tensor([L, 0, 0, L, 0, L], dtype=torch.int32).cuda()
    for act in (pnr.ACT_NONE, pnr.ACT_SILU):
        kw = dict(weight=w, bias=b, gate=gate if gated else None, act=act, lens=lens)
        f = pnr.group_norm(x, 2, **kw)
        d = pnr.group_norm_backward(gy, x, 2, f["mean"], f["rstd"], **kw)
        for t in [f["y"], d["x"]] + ([d["gate"]] if gated else []):
            assert (t[lens == 0] == 0).all()
