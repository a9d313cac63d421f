"""Checks of the sequence-mixing binding that need no GPU."""
import pytest
import torch

from nonlinear_rnn_evaluation_amd import pnr


@pytest.mark.parametrize("ws", [torch.empty(1, dtype=torch.uint8).expand(4096), torch.empty(8192, dtype=torch.uint8)[::2]],
                         ids=["expanded", "strided"])
def test_a_workspace_covers_its_bytes(ws):
    """The library is told the tensor's number of bytes: they have to be there, one after the other."""
    desc = pnr.PnrNorm()
    with pytest.raises(ValueError, match="contiguous"):
        pnr._workspace(4096, ws, ws.get_device(), desc)


def test_sizes_beyond_the_descriptor_are_named():
    x = torch.empty(2, 3, 8)
    with pytest.raises(pnr.PnrError, match="32 bits"):
        pnr._pack(pnr.PnrNorm, pnr._NORM, *x.shape, 2 ** 31, pnr.F32, pnr.ACT_NONE, 1e-5, 0, 0, 0, 0)
    d = pnr._pack(pnr.PnrNorm, pnr._NORM, *x.shape, 4, pnr.F32, pnr.ACT_SILU, 1e-5, 0, 0, 0, 0)
    assert (d.N, d.L, d.C, d.groups, d.dtype, d.act, d.eps) == (2, 3, 8, 4, pnr.F32, pnr.ACT_SILU, 1e-5)
