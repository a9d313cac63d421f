"""The mixed layer (nonlinear_rnn_evaluation_amd/mixer.py) end to end: prompts against single tokens,
its gradients against differences of its output, and its forward pass against the fp64 oracles."""
import numpy as np
import pytest
import torch

import oracle as O
from nonlinear_rnn_evaluation_amd import mixer, pnr
from nonlinear_rnn_evaluation_amd import workloads as WL


def _layer(D=48, H=4, H_kv=2, Dk=16, Dv=24):
    return mixer.Mixer(D, H, H_kv, Dk, Dv, seed=3)


def _x(B, T, D, seed=4):
    return torch.randn(B, T, D, generator=torch.Generator().manual_seed(seed)).cuda()


def _reference(m, x, lens=None):
    """The layer in fp64 on the oracles."""
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    B, T, D = x.shape
    h = O.sequential(WL.CELL_GRU_DIAG, d(m.W), d(m.U), None, None, d(x), np.zeros((B, D)))
    q, k, v, gate, a = np.split(h @ d(m.W_in), np.cumsum(m.sizes)[:-1], -1)
    o, S = O.linear_attention(q.reshape(B, T, m.H, m.Dk), k.reshape(B, T, m.H_kv, m.Dk), v.reshape(B, T, m.H_kv, m.Dv),
                              -np.log1p(np.exp(-(a + 3.0))), m.Dk ** -0.5, None, lens)
    C = m.H * m.Dv
    y, _, _ = O.group_norm(o.reshape(B * T, 1, C), m.H, d(m.norm_w), d(m.norm_b), gate.reshape(B * T, 1, C), "silu")
    return y.reshape(B, T, C) @ d(m.W_out), S


@pytest.mark.gpu
def test_prompts_against_the_oracles():
    m, x = _layer(), _x(3, 150, 48)
    lens = torch.tensor([150, 64, 1], dtype=torch.int32).cuda()
    r = m.prompt(x, lens)
    out, S = _reference(m, x, lens.cpu().numpy())
    for b, n in enumerate(lens.tolist()):
        assert np.abs(r["out"][b, :n].double().cpu().numpy() - out[b, :n]).max() <= 1e-4 * np.abs(out).max()
    assert np.abs(r["S"].double().cpu().numpy() - S).max() <= 1e-4 * np.abs(S).max()


@pytest.mark.gpu
def test_tokens_continue_a_prompt():
    m, x = _layer(), _x(2, 40, 48)
    whole = m.prompt(x)
    part = m.prompt(x[:, :30].contiguous())
    pool, slots = torch.zeros(5, 2, 16, 24, device="cuda"), torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = part["S"]
    h = part["h"].contiguous()
    for t in range(30, 40):
        out, h = m.token(x[:, t].contiguous(), h, pool, slots)
        assert (out - whole["out"][:, t]).abs().max() <= 1e-4 * whole["out"].abs().max()
    assert (pool[slots.long()] - whole["S"]).abs().max() <= 1e-4 * whole["S"].abs().max()


@pytest.mark.gpu
def test_gradients_against_differences():
    """Along one random direction of each argument: fp32 differences of a loss of size ~1, so
    a step of 1e-2 and 1 % of the larger of the two sides."""
    m, x = _layer(), _x(2, 70, 48)
    grad_out = torch.randn(x.shape, generator=torch.Generator().manual_seed(9)).cuda() / x.numel() ** 0.5
    g = m.gradients(x, grad_out)
    assert (g["out"] - m.prompt(x)["out"]).abs().max() <= 1e-5 * g["out"].abs().max()
    for name in ("x", "W", "U", "W_in", "W_out", "norm_w", "norm_b"):
        p = x if name == "x" else getattr(m, name)
        v = torch.randn(p.shape, generator=torch.Generator().manual_seed(11)).cuda()
        v = v + 3 * g[name] / g[name].norm() * v.norm()          # a direction along which the loss changes
        v = v / v.norm()
        loss = []
        for s in (1e-2, -1e-2):
            p.add_(s * v)
            loss.append((m.prompt(x)["out"].double() * grad_out.double()).sum().item())
            p.sub_(s * v)
        diff, want = (loss[0] - loss[1]) / 2e-2, (g[name].double() * v.double()).sum().item()
        print(f"# {name}: {diff:.6f} {want:.6f}", flush=True)
        assert abs(diff - want) <= 1e-2 * max(abs(diff), abs(want)), (name, diff, want)


@pytest.mark.gpu
def test_the_example_runs(capsys):
    mixer.main()
    said = capsys.readouterr().out
    assert "largest difference" in said and "training loss" in said
    loss = [float(v) for v in said.split("training loss:")[1].split()]
    assert all(np.isfinite(loss)) and loss[-1] < loss[0]
