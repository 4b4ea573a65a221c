"""CPU: the sequence operators' host code under AddressSanitizer and UndefinedBehaviorSanitizer, driven through
every size query and argument-error path (tests/host_sanitize/driver_sequence.cpp).  Nothing reaches the GPU."""
import os
import shutil
import subprocess

import pytest

from tests import test_host_sanitize as base

DRIVER = os.path.join(base.ROOT, "tests", "host_sanitize", "driver_sequence.cpp")


@pytest.mark.skipif(base._hipcc() is None or shutil.which("ld") is None, reason="needs hipcc")
def test_sequence_operators_under_the_sanitizers():
    base._build()  # the library's objects
    main = base._compile((DRIVER, os.path.join(base.OUT, "driver_sequence.o"), []))
    objs = [os.path.join(base.OUT, os.path.splitext(os.path.basename(s))[0] + ".o") for s in base._sources()]
    exe = os.path.join(base.OUT, "driver_sequence")
    link = subprocess.run([base._hipcc(), f"--offload-arch={base.libbuild.ARCH}", *base.HOST_SAN, main, *objs, "-o", exe,
                           *base.libbuild.LIBS], capture_output=True, text=True)
    assert link.returncode == 0, link.stdout + link.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    text = res.stdout + res.stderr
    assert res.returncode == 0, text
    assert "runtime error" not in text and "Sanitizer" not in text, text
    assert "failures 0" in res.stdout, text
