"""Every launch of the layer norm and the embedding, over the documented range
of sizes, stays within HIP's limit of 2^32 - 1 work-items.  Host only: the
launches are recorded (launch_recorder.c) and none runs."""
import json
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

# run in a process of its own, with the recorder loaded before the HIP runtime
PROGRAM = r"""
import ctypes, json, sys
rec = ctypes.CDLL(sys.argv[1])
rec.recorded_launches.restype = rec.recorded_largest.restype = ctypes.c_uint64
sys.path.insert(0, sys.argv[2])
import stable_variance_amd as sv
L = sv.capi()
P = ctypes.c_void_p(0x1000)  # never dereferenced
out = []

def call(what, fn, *args):
    rec.recorded_clear()
    status = fn(*args)
    out.append([what, status, rec.recorded_launches(), rec.recorded_largest(),
                L.sv_last_error_message().decode() if status else ""])

for dtype in (0, 1, 2):
    lengths = [1, 3, 64, 1531, 4096, 16384, 20001, 1 << 20, (1 << 27) - 64, (1 << 27) - 63, (1 << 27) - 1, 1 << 27]
    for n in lengths:
        for rows in sorted({1, 3, 70000, min(1 << 28, (1 << 36) // n), (1 << 36) // n}):
            if rows * n > 1 << 36:
                continue
            call(f"norm {dtype} {rows} {n}", L.sv_layer_norm, P, dtype, rows, n, n, None, None, 0, 1e-5, P, n, P, P, None)
            need = L.sv_layer_norm_backward_workspace_size(rows, n, dtype)
            for dw, db in ((P, P), (P, None), (None, P), (None, None)):
                call(f"norm gradient {dtype} {rows} {n} {dw} {db}", L.sv_layer_norm_backward, P, n, P, n, dtype, rows,
                     n, None, 0, P, P, P, n, dw, db, P, need, None)
    for dim in (1, 3, 8, 64, 257, 4096, 1 << 20, 1 << 27):
        most = (1 << 36) // dim
        for tokens in sorted({1, 1000, 5000, 70000, min(most, 1 << 30)}):
            for vocab in sorted({1, 300, 64000, min(most, (1 << 31) - 2)}):
                if tokens > most or vocab > most:
                    continue
                call(f"lookup {dtype} {tokens} {vocab} {dim}", L.sv_embedding, P, 8, tokens, P, dtype, vocab, dim, dim,
                     1.0, P, dim, None)
                need = L.sv_embedding_backward_workspace_size(tokens, vocab, dim, dtype)
                call(f"lookup gradient {dtype} {tokens} {vocab} {dim}", L.sv_embedding_backward, P, dim, P, 8, tokens,
                     dtype, vocab, dim, 1.0, -1, P, dim, P, need, None)
# the knob that lowers the limit reaches the join of the column sums
sv.set_tuning("launch_items", 1024)
need = L.sv_layer_norm_backward_workspace_size(8, 1000, 0)
call("knob", L.sv_layer_norm_backward, P, 1000, P, 1000, 0, 8, 1000, None, 0, P, P, None, 1000, P, P, P, need, None)
print(json.dumps(out))
"""


def test_every_launch_is_within_the_limit(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    so = str(tmp_path / "launch_recorder.so")
    res = subprocess.run([gcc, "-O1", "-Wall", "-Werror", "-shared", "-fPIC", os.path.join(HERE, "launch_recorder.c"),
                          "-o", so], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    # before whatever else is preloaded here
    pre = " ".join(p for p in (so, os.environ.get("LD_PRELOAD", "")) if p)
    res = subprocess.run([sys.executable, "-c", PROGRAM, so, os.path.dirname(HERE)], capture_output=True, text=True,
                         timeout=600, env={**os.environ, "LD_PRELOAD": pre})
    assert res.returncode == 0, res.stderr[-4000:]
    calls = json.loads(res.stdout.strip().splitlines()[-1])
    assert len(calls) > 500
    bad = [c for c in calls if c[1] != 0 or c[3] > 0xffffffff]
    assert not bad, bad[:10]
    assert all(c[2] > 0 for c in calls)  # the recorder saw the launches
    # 16 + 16 tiles of 64 columns, one workgroup of 1024 threads per launch
    assert calls[-1][0] == "knob" and calls[-1][2] == 1 + 32, calls[-1]
