"""Group norm on many maps, wide groups and rows off a vector's alignment: the workspace stays bounded in the
number of rows, and the gradients of weight and bias add up over all of them.

Tolerances as test_gpu_groupnorm.py derives them: 2 * 2^-9 of the norm for bf16 outputs, 2^-17 for fp32 ones."""
import os

import numpy as np
import pytest
import torch

import oracle as O
from nonlinear_rnn_evaluation_amd import pnr

BF16, F32 = torch.bfloat16, torch.float32
TOL = {BF16: 2 * 2.0 ** -9, F32: 2.0 ** -17}
BOUND = 64 << 20


def _sizes(N, L, C, groups, dtype):
    d = pnr.PnrNorm(N, L, C, groups, dtype, pnr.ACT_NONE, 1e-5)
    return pnr.pnr_groupnorm_workspace_bytes(d), pnr.pnr_groupnorm_workspace_bytes_backward(d)


@pytest.mark.skipif(not os.path.exists(pnr.LIB_PATH), reason="libpnr.so not built")
@pytest.mark.parametrize("dtype", [pnr.BF16, pnr.F32])
@pytest.mark.parametrize("L,C,groups", [(1, 1024, 1), (1, 4096, 1), (1, 8192, 1), (1, 513, 1), (1, 6000, 2), (1, 20000, 1),
                                        (2, 2048, 16), (2, 64, 64), (3, 33, 11), (300, 320, 32)])
def test_the_workspace_does_not_grow_with_the_rows(L, C, groups, dtype):
    few, many = _sizes(1 << 12, L, C, groups, dtype), _sizes(1 << 16, L, C, groups, dtype)
    for a, b in zip(few, many):
        assert b <= max(BOUND + (1 << 20), a), (few, many)


def _near(name, got, ref, tol):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    err, norm = np.linalg.norm(got - ref), np.linalg.norm(ref)
    print(f"#   {name}: {err / norm:.2e} (tol {tol:.1e})", flush=True)
    assert err <= tol * norm, (name, err, norm)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("aligned", [True, False], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("N,L,C,groups", [
    # more rows than one batch of the workspace takes (the first), wide groups of tokens, short maps
    (2500, 1, 5000, 1), (1500, 1, 6000, 1), (700, 1, 9001, 1), (9000, 2, 513, 1), (3000, 1, 513, 1), (5, 1, 8192, 1), (900, 3, 4800, 16)])
def test_many_rows(N, L, C, groups, aligned, dtype):
    gen = torch.Generator().manual_seed(N)
    draw = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    off = 0 if aligned else 1

    def rows():
        return draw(N * L * C + off).to(dtype).cuda()[off:].view(N, L, C)
    x, gy, gate = rows(), rows(), rows()
    w, b = (1 + 0.3 * draw(C)).cuda(), (0.3 * draw(C)).cuda()
    lens = torch.tensor([(L, 0, L)[i % 3] for i in range(N)], dtype=torch.int32).cuda()
    kw = dict(weight=w, bias=b, gate=gate, act=pnr.ACT_SILU, lens=lens)
    f = pnr.group_norm(x, groups, **kw)
    d = pnr.group_norm_backward(gy, x, groups, f["mean"], f["rstd"], **kw)
    X, Y, G, W, Bb = (t.double().cpu().numpy() for t in (x, gy, gate, w, b))
    ref = (groups, W, Bb, G, "silu", 1e-5, lens.cpu().numpy())
    y, mean, rstd = O.group_norm(X, *ref)
    _near("y", f["y"], y, TOL[dtype])
    _near("rstd", f["rstd"], rstd, TOL[F32])
    g = O.group_norm_grad(Y, X, *ref)
    _near("grad_x", d["x"], g["x"], TOL[dtype] * (1 if dtype == BF16 else 4))
    _near("grad_gate", d["gate"], g["gate"], TOL[dtype])
    _near("grad_weight", d["weight"], g["weight"], TOL[F32])
    _near("grad_bias", d["bias"], g["bias"], TOL[F32])
    only = pnr.group_norm_backward(gy, x, groups, f["mean"], f["rstd"], want=("bias",), **kw)
    assert torch.equal(only["bias"], d["bias"])
