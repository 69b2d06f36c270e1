"""Host code of the norm and of the packed serving step's operators under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): tests/host_sanitize/packed.cpp calls their argument
validation with sizes at the ends of the integer types."""

import os
import subprocess

import pytest

from binary_coded_precision_amd import build as hb
from test_lowbit_sanitizers import ENV, HERE


def test_validation_is_clean_under_asan_and_ubsan():
    try:
        driver = hb.build_host_sanitized(os.path.join(HERE, "host_sanitize", "packed.cpp"))
    except RuntimeError as e:  # a toolchain without the sanitizer runtimes
        pytest.skip("sanitized host build unavailable: %s" % str(e)[:200])
    r = subprocess.run([driver], capture_output=True, text=True, timeout=120, env=ENV)
    assert "AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[-2000:]
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    assert r.stdout.strip().endswith("0 failures")
