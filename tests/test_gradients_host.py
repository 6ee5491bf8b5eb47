"""Clipping's search for overlaps without host memory."""
import os
import subprocess
import sys

import stable_variance_amd as sv

PROGRAM = r"""
import ctypes, resource, sys
sys.path.insert(0, sys.argv[1])
import stable_variance_amd as sv
L = sv.capi()
n = 1 << 20
ptrs = (ctypes.c_void_p * n)(*range(1 << 32, (1 << 32) + n * 64, 64))  # never dereferenced
sizes, codes = (ctypes.c_int64 * n)(*[1] * n), (ctypes.c_int * n)()
need = L.sv_grad_norm_workspace_size(sizes, codes, n)
P = ctypes.c_void_p(0x10000)

def clip():
    # the workspace is looked at behind the search
    return L.sv_clip_grad_norm(ptrs, ptrs, sizes, codes, n, 1.0, P, P, need - 1, None), L.sv_last_error_message()

status, message = clip()
assert status == 2, (status, message)
with open("/proc/self/statm") as f:
    used = int(f.read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (8 << 20), resource.RLIM_INFINITY))  # the search takes 48 MB
print(*clip())
"""


def test_no_host_memory_is_not_the_arguments_fault():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", PROGRAM, root], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-4000:]
    assert res.stdout.split(None, 1) == ["6", "b'sv_clip_grad_norm: no host memory for 1048576 tensors'\n"]
    assert sv.capi().sv_status_string(6) == b"SV_ERR_HOST_MEMORY"
    assert "SV_ERR_HOST_MEMORY" in str(sv.SvError(6, ""))
