"""Linear attention in bf16: an output is the 64-bit result rounded once, but for what fp32 inside loses.

The bar, as the 2-norm of (output - rounded 64-bit result) over the result's: let the value before its
rounding be off by a vector d of norm e times the result's.  An element changes its rounding with a
probability of |d_i| / ulp_i, and then by ulp_i, so the squared difference is sum |d_i| ulp_i
<= |d| |ulp|, and ulp_i <= 2^-7 |x_i|: a difference of sqrt(2^-7 e).  Operands as two bf16 parts are off by at
most 2^-17 each (the second part's rounding, of a remainder of up to 2^-8); with two such operands and the
fp32 sums e <= 2^-15, a bar of 2^-11.  One rounding of an operand to bf16 (2^-9) shows as 2^-8.6.
"""
import numpy as np
import pytest
import torch

import oracle as O
from nonlinear_rnn_evaluation_amd import pnr

BAR = 2.0 ** -11

SHAPES = [
    # B, T, H, Hkv, Dk, Dv: one chunk, several chunks of one block, segments, shared heads, unaligned rows
    (1, 37, 8, 8, 64, 64), (2, 64, 4, 2, 128, 128), (1, 250, 2, 2, 128, 128), (2, 333, 4, 2, 64, 128),
    (1, 700, 2, 1, 128, 64), (1, 200, 5, 1, 100, 72), (1, 90, 2, 2, 33, 17), (40, 400, 8, 8, 16, 24),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_bf16_outputs_are_rounded_once(shape):
    B, T, H, Hkv, Dk, Dv = shape
    gen = torch.Generator().manual_seed(SHAPES.index(shape))
    draw = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k, v, go = (draw(B, T, h, d).bfloat16().cuda() for h, d in ((H, Dk), (Hkv, Dk), (Hkv, Dv), (H, Dv)))
    g = -torch.empty(B, T, Hkv).exponential_(20.0, generator=gen).cuda()        # a memory of some twenty tokens
    state, gs = draw(B, Hkv, Dk, Dv).cuda(), draw(B, Hkv, Dk, Dv).cuda()
    kw = dict(scale=Dk ** -0.5, state=state)
    got = {"o": pnr.linear_attention(q, k, v, g, **kw)["o"]}
    got.update(pnr.linear_attention_backward(q, k, v, g, go, grad_state=gs, **kw))
    q, k, v, g, go, state, gs = (t.double().cpu().numpy() for t in (q, k, v, g, go, state, gs))
    ref = O.linear_attention_grad(q, k, v, g, Dk ** -0.5, go, state, None, gs)
    ref["o"] = O.linear_attention(q, k, v, g, Dk ** -0.5, state)[0]
    for n in ("o", "q", "k", "v"):
        once = torch.from_numpy(ref[n]).bfloat16().double().numpy()
        err = np.linalg.norm(got[n].double().cpu().numpy() - once) / np.linalg.norm(ref[n])
        print(f"# {shape} {n}: {err:.2e} (bar {BAR:.1e})", flush=True)
        assert err <= BAR, (n, err)
