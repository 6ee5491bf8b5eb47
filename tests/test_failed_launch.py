"""Clipping whose launches fail, on the host: tensors are not scaled by a factor
that no kernel has written."""
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

PROGRAM = r"""
import ctypes, sys
stub = ctypes.CDLL(sys.argv[1])
launches, fail_at = (ctypes.c_int.in_dll(stub, name) for name in ("launches", "fail_at"))
sys.path.insert(0, sys.argv[2])
import stable_variance_amd as sv
L = sv.capi()
n = 300  # three launches of the sum, one of the join, three of the scaling
ptrs = (ctypes.c_void_p * n)(*range(1 << 20, (1 << 20) + n * 256, 256))  # never dereferenced
sizes, codes = (ctypes.c_int64 * n)(*[5] * n), (ctypes.c_int * n)()
need = L.sv_grad_norm_workspace_size(sizes, codes, n)
P = ctypes.c_void_p(0x10000)
for at in range(8):
    launches.value, fail_at.value = 0, at
    status = L.sv_clip_grad_norm(ptrs, ptrs, sizes, codes, n, 1.0, P, P, need, None)
    print(at, status, launches.value)
"""


def test_nothing_is_scaled_without_a_factor(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    so = str(tmp_path / "failing_launch.so")
    res = subprocess.run([gcc, "-O1", "-Wall", "-Werror", "-shared", "-fPIC", os.path.join(HERE, "failing_launch.c"),
                          "-o", so], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    # before whatever else is preloaded here
    pre = " ".join(p for p in (so, os.environ.get("LD_PRELOAD", "")) if p)
    res = subprocess.run([sys.executable, "-c", PROGRAM, so, os.path.dirname(HERE)], capture_output=True, text=True,
                         timeout=300, env={**os.environ, "LD_PRELOAD": pre})
    assert res.returncode == 0, res.stderr[-4000:]
    got = {at: (status, launches) for at, status, launches in
           (map(int, line.split()) for line in res.stdout.strip().splitlines())}
    for at in range(4):  # the sum or the join: the scaling is not launched
        assert got[at][0] == 4 and got[at][1] <= 4, (at, got[at])
    for at in range(4, 7):
        assert got[at][0] == 4, (at, got[at])
    assert got[7] == (0, 7)
