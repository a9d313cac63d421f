"""What the single-token calls do not read they do not refuse either (no GPU: the calls end at a later argument)."""
import os

import pytest

from nonlinear_rnn_evaluation_amd import pnr
from test_abi_selscan import P, _conv, _forward, _scan, _step

pytestmark = pytest.mark.skipif(not os.path.exists(pnr.LIB_PATH), reason="libpnr.so not built")


@pytest.mark.parametrize("lens", [P + 1, P + 2, 3])
def test_row_lengths(lens):
    d = _scan()
    d.lens = lens
    assert _forward(d) == pnr.E_INVALID and "aligned" in pnr.pnr_last_error()
    assert _step(d, y=None) == pnr.E_INVALID and "y is NULL" in pnr.pnr_last_error()
    d = _conv()
    d.lens = lens
    assert pnr.pnr_conv_forward(d, P, None, P, None, None, P, None) == pnr.E_INVALID and "aligned" in pnr.pnr_last_error()
    assert pnr.pnr_conv_step(d, P, P, None, P, None, 2, None, P) == pnr.E_INVALID and "y is NULL" in pnr.pnr_last_error()
