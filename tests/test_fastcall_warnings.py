"""The call module compiles without a warning: one of them would hide that it
names something that the library's header names too."""
import os
import subprocess
import sysconfig

import pytest

from zero_collectives_gb300 import build


def test_no_warnings():
    inc = sysconfig.get_paths().get("include") or ""
    if not os.path.exists(os.path.join(inc, "Python.h")):
        pytest.skip("no Python headers")
    src = os.path.join(build.CSRC, "fastcall.c")
    try:
        r = subprocess.run([os.environ.get("CC", "cc"), "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-I", inc, "-I", build.INCLUDE, src],
                           capture_output=True, text=True)
    except OSError:
        pytest.skip("no C compiler")
    assert r.returncode == 0, r.stderr
