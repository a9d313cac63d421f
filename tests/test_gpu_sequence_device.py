"""The sequence-mixing calls launch on their tensors' device, whichever one is current: on one device this
shows by the device that the binding selects around each call."""
import contextlib

import pytest
import torch

from nonlinear_rnn_evaluation_amd import pnr


@pytest.mark.gpu
def test_calls_select_their_tensors_device(monkeypatch):
    q, k, v = (torch.randn(2, 8, 2, 16, device="cuda") for _ in range(3))
    g = torch.full((2,), -0.1, device="cuda")
    x = torch.randn(4, 1, 32, device="cuda")
    dev = q.get_device()

    def calls():
        a = pnr.linear_attention(q, k, v, g)
        b = pnr.linear_attention_backward(q, k, v, g, a["o"])
        c = pnr.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g, a["state"].clone())
        n = pnr.group_norm(x, 4)
        d = pnr.group_norm_backward(x, x, 4, n["mean"], n["rstd"])
        return [a["o"], a["state"], b["q"], b["log_decay"], c["o"], c["state"], n["y"], d["x"]]
    ref, seen = calls(), []

    @contextlib.contextmanager
    def select(device):
        seen.append(device)
        yield
    monkeypatch.setattr(torch.cuda, "device", select)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: dev)
    calls()
    assert seen == []                       # the current device needs no selection
    monkeypatch.setattr(torch.cuda, "current_device", lambda: dev + 1)
    for p, q_ in zip(ref, calls()):
        assert torch.equal(p, q_)
    assert seen == [dev] * 5


@pytest.mark.gpu
def test_a_refused_number_of_groups_allocates_nothing_for_them():
    x = torch.zeros(2, 3, 12, device="cuda")
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(pnr.PnrError, match="divide"):
        pnr.group_norm(x, 10 ** 7)
    assert torch.cuda.max_memory_allocated() - before < 1 << 20
