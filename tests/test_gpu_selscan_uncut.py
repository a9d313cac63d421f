"""The selective scan where rows fill the device, so that time is in one piece, against the fp64 oracle and against
calls that cut it: gradients of every state count and both types over rows that end early, prompts of many states,
row lengths that say what their absence says.

Time is in one piece backwards from 2048 waves on, a wave for 64 channels of one group and 16 states, and forwards
from 1280 waves of 16 channels on, 4096 where rows have lengths; the shapes below are chosen for that.
"""
import pytest
import torch

from nonlinear_rnn_evaluation_amd import pnr
from test_gpu_selscan import BF16, F32, TOKENS, TOL, _case, _check, _f64, _near, _split


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(32, 70, 512, 16, 64), (16, 70, 512, 24, 64), (11, 70, 520, 33, 65), (8, 70, 512, 64, 64),
                                   (32, 37, 4096, 16, 1), (33, 70, 128, 5, 64)], ids=str)
def test_gradients_of_rows_that_end_early(shape, dtype):
    B, T, E, N, G = shape
    assert B * G * (((E // G) + 63) // 64) * ((N + 15) // 16) >= 2048
    lens = ([T, 0, 1, 16, 17, T - 1, 33, T + 5, -1, 15, 32] * 3)[:B]
    _check(*_case(80, B, T, E, N, G, dtype, gated=N != 24, softplus=N != 33, lens=lens))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [16, 24, 33, 64])
def test_gradients_of_a_batch_are_its_rows(N, dtype):
    """Several chunks a row; the same rows alone are cut."""
    B, T, E, G = 2048 // 64 // ((N + 15) // 16) + 1, 150, 512, 64
    c, gy, gs = _case(81, B, T, E, N, G, dtype, lens=([T, 0, 1, 16, 64, 149] * 6)[:B])
    args, kw = _split(c)
    d = pnr.selective_scan_backward(*args, gy, grad_state=gs, **kw)
    for b in (0, 1, 2, 3, 4, 5, B - 1):
        one = [a if a.dim() == 2 else a[b:b + 1] for a in args]
        row = {k: v[b:b + 1] if k in ("z", "state", "lens") else v for k, v in kw.items()}
        r = pnr.selective_scan_backward(*one, gy[b:b + 1], grad_state=gs[b:b + 1], **row)
        for n in TOKENS + ("state",):
            _near(f"{n} of row {b}", d[n][b], _f64(r[n][0]), 2 * (TOL[dtype] if n in TOKENS else TOL[F32]))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [40, 64])
def test_prompts_of_many_states(N):
    """Six rows of 256 waves in one pass, a row alone in two."""
    c, _, _ = _case(82, 6, 300, 4096, N, 1, BF16)
    args, kw = _split(c)
    got = pnr.selective_scan(*args, **kw)
    assert got["workspace"] is None or got["workspace"].numel() == 0
    for b in (0, 5):
        row = {k: v[b:b + 1] if k in ("z", "state") else v for k, v in kw.items()}
        r = pnr.selective_scan(*[a if a.dim() == 2 else a[b:b + 1] for a in args], **row)
        assert r["workspace"].numel() > 0
        _near("y", got["y"][b], _f64(r["y"][0]), 2 * TOL[BF16])
        _near("state", got["state"][b], _f64(r["state"][0]), 2 * TOL[F32])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_lengths_of_all_tokens_are_no_lengths(dtype):
    """1792 waves: one pass without lengths, two with."""
    c, gy, gs = _case(83, 7, 600, 4096, 16, 1, dtype)
    args, kw = _split(c)
    plain = pnr.selective_scan(*args, **kw)
    d = pnr.selective_scan_backward(*args, gy, grad_state=gs, **kw)
    kw["lens"] = torch.full((7,), 600, dtype=torch.int32, device="cuda")
    full = pnr.selective_scan(*args, **kw)
    _near("y", full["y"], _f64(plain["y"]), 2 * TOL[dtype])
    _near("state", full["state"], _f64(plain["state"]), 2 * TOL[F32])
    e = pnr.selective_scan_backward(*args, gy, grad_state=gs, **kw)
    for n in d:
        if n != "workspace":
            assert torch.equal(d[n], e[n]), n
