"""Host memory that runs out inside a C entry of the 4-bit block products is
reported like any other error.  In a process of its own, whose operator new is
replaced by one that fails when told to."""

import os
import shutil
import subprocess
import sys

import pytest

pytest.importorskip("newton_schulz_dmuon_amd")
from newton_schulz_dmuon_amd import _lib  # noqa: E402
from test_q8_no_memory import NEW  # noqa: E402

CALLS = """
import ctypes, sys
new = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
from newton_schulz_dmuon_amd import _lib
lib = _lib.load()
a = [0x7F0000000000 + i * 0x100000000 for i in range(6)]
m = (_lib.Q4SourceDesc * 1)(_lib.Q4SourceDesc(a[0], _lib.BF16, 0, 256, 128, None, a[1], a[2], a[3], a[4]))
calls = [lambda: lib.dmuon_q4_quantize(m, 1, None),
         lambda: lib.dmuon_q4_dequantize(a[0], a[1], 4, 256, a[2], _lib.BF16, None),
         lambda: lib.dmuon_q4_matmul(a[0], a[1], 8, a[2], a[3], 256, 512, None, a[4], _lib.BF16, a[5], 1 << 40, None),
         lambda: lib.dmuon_q4_rows_matmul(a[0], 8, a[2], a[3], 256, 512, a[4], _lib.BF16, a[5], 1 << 40, None)]
for call in calls:
    new.set_failing(1)
    status = call()
    new.set_failing(0)
    print(status, lib.dmuon_last_error().decode())
"""


def test_a_failed_allocation_is_an_error(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    source, lib = tmp_path / "new.cpp", tmp_path / "new.so"
    source.write_text(NEW)
    subprocess.run([cxx, "-shared", "-fPIC", "-O1", str(source), "-o", str(lib)], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(_lib.__file__)))
    run = subprocess.run([sys.executable, "-c", CALLS, str(lib), root], capture_output=True, text=True, timeout=100)
    assert run.returncode == 0, run.stderr[-500:]
    assert run.stdout.split("\n") == [f"{_lib.ERR_INVALID_ARG} internal error: std::bad_alloc"] * 4 + [""]
