"""Edge calls of the layer operators that end on the host (CPU only: no call
here reaches a kernel launch)."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# In a process of its own: an integer division by zero ends the interpreter.
QUERY = """
import ctypes, os, sys
sys.path.insert(0, sys.argv[1])
from depthwise_causal_conv1d_amd import _lib
if not os.path.exists(_lib.LIB_PATH):
    from depthwise_causal_conv1d_amd import build
    build.build()
f, b = ctypes.c_int64(-1), ctypes.c_int64(-1)
rc = _lib.load().gated_linear_recurrence_workspace(int(sys.argv[2]), int(sys.argv[3]), 0,
                                                   ctypes.byref(f), ctypes.byref(b))
print(rc, f.value, b.value)
"""


@pytest.mark.parametrize("total_T,batch", [(0, 0), (0, 3), (100, 1), (200, 1), (1000, 1), (1000, 4),
                                           ((1 << 31) - 4097, 1)])
def test_recurrence_workspace_without_channels(total_T, batch):
    """dim == 0 is a no-op of both packed calls, and needs no workspace."""
    got = subprocess.run([sys.executable, "-c", QUERY, ROOT, str(total_T), str(batch)],
                         capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stderr[-500:]
    assert got.stdout.split() == ["0", "0", "0"]
