"""The state space layer rounds what it keeps only when asked to: gradients without a choice are the exact ones."""
import pytest
import torch

from nonlinear_rnn_evaluation_amd import mixer


@pytest.mark.gpu
def test_nothing_is_rounded_unasked():
    m = mixer.StateSpace(24, 72, G=2, seed=3)
    g = torch.Generator().manual_seed(8)
    x, grad_out = torch.randn(2, 50, 24, generator=g).cuda(), torch.randn(2, 50, 24, generator=g).cuda()
    plain, exact, kept = m.gradients(x, grad_out), m.gradients(x, grad_out, keep=False), m.gradients(x, grad_out, keep=True)
    assert torch.equal(plain["conv_w"], exact["conv_w"]) and torch.equal(plain["A_log"], exact["A_log"])
    assert not torch.equal(kept["conv_w"], exact["conv_w"])
