"""The host code of the sequence-mixing entry points under AddressSanitizer and UndefinedBehaviorSanitizer, as
tests/test_host_sanitized.py does it for the others.  No device call is made: this runs on the CPU."""
import os
import subprocess
import sys

import pytest

from nonlinear_rnn_evaluation_amd.build import LIB_SANITIZED, build_library
from test_host_sanitized import ROOT, _asan_runtime, _stale


@pytest.mark.skipif(_asan_runtime() is None, reason="no AddressSanitizer runtime in this toolchain")
def test_sequence_mixing_host_code_under_sanitizers():
    if _stale(LIB_SANITIZED):
        build_library(sanitize=True)
    env = dict(os.environ, LD_PRELOAD=_asan_runtime(), ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:exitcode=23",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1:exitcode=24")
    out = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "host_sanitized_sequence.py"), LIB_SANITIZED],
                         env=env, capture_output=True, text=True, timeout=600)
    report = out.stdout + out.stderr
    assert "AddressSanitizer" not in report and "runtime error:" not in report, report[-4000:]
    assert out.returncode == 0 and "host checks passed" in out.stdout, report[-4000:]
