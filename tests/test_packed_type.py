"""A packed activation knows the type it was made of: causal_conv of it gives that type, and asks where nobody said."""
import copy
import pickle

import pytest
import torch

from nonlinear_rnn_evaluation_amd import pnr


def test_a_packed_activation_is_a_pair_that_keeps_its_type():
    codes, exps = torch.zeros(2, 3, 40, dtype=torch.int8), torch.ones(2, 3, 2, dtype=torch.uint8)
    p = pnr.Packed(codes, exps, torch.float32)
    a, b = p
    assert a is codes and b is exps and len(p) == 2 and p.dtype == torch.float32
    assert copy.copy(p).dtype == torch.float32 and pickle.loads(pickle.dumps(p)).dtype == torch.float32
    assert pnr.Packed(codes, exps).dtype is None and p._replace(codes=codes).dtype is None


def test_a_type_that_nobody_said_is_asked_for():
    p = pnr.Packed(torch.zeros(2, 3, 40, dtype=torch.int8), torch.ones(2, 3, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="dtype"):
        pnr.causal_conv(p, torch.zeros(40, 4))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_the_convolution_of_a_copy_has_its_type(dtype):
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(2, 50, 40, generator=g).to(dtype).cuda(), torch.randn(40, 4, generator=g).cuda()
    p = pnr.checkpoint_pack(x)
    assert p.dtype == dtype
    got, want = pnr.causal_conv(p, w), pnr.causal_conv(pnr.checkpoint_unpack(p, dtype), w)
    assert got["y"].dtype == got["state"].dtype == dtype
    assert torch.equal(got["y"], want["y"]) and torch.equal(got["state"], want["state"])
    other = torch.bfloat16 if dtype == torch.float32 else torch.float32
    assert pnr.causal_conv(p, w, dtype=other)["y"].dtype == other
