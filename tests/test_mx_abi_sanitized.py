"""The argument checks of the MXFP4 quantisation, the products and the expert layer under host sanitizers:
their ABI tests against the build of the C-ABI layer that test_abi_sanitized makes.  No GPU needed."""
import os
import shutil
import subprocess
import sys

import pytest

from conftest import ROOT
from test_abi_sanitized import _runtime


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_mx_abi_under_host_sanitizers():
    asan, ubsan = _runtime("libasan.so"), _runtime("libubsan.so")
    if not (asan and ubsan):
        pytest.skip("sanitizer runtimes not installed")
    from mxfp4_mixture_experts_amd import build_lib
    lib = build_lib.build_host_sanitized()
    env = dict(os.environ)
    env.update({
        "MXFP4_MOE_LIB": lib,
        "LD_PRELOAD": f"{asan} {ubsan}",
        # the interpreter and the HIP runtime keep allocations until exit: leaks are not this layer's
        "ASAN_OPTIONS": "detect_leaks=0:abort_on_error=1",
        "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1",
        "HIP_VISIBLE_DEVICES": "",
    })
    files = [os.path.join(ROOT, "tests", f) for f in ("test_mx_abi.py", "test_mx_layer_abi.py")]
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", *files],
                         capture_output=True, text=True, env=env, cwd=ROOT, timeout=600)
    text = res.stdout + res.stderr
    assert res.returncode == 0, text[-4000:]
    assert "AddressSanitizer" not in text and "runtime error" not in text, text[-4000:]
    assert " passed" in text and "skipped" not in text
