"""The module that takes ordinary tensors to the library: what it does when a
launch fails, and whether other threads run meanwhile.

A process of its own loads a stand-in for the library's calls before the
module (tests/library_stand_in.c).  The stand-in launches nothing; the Python
functions' general way reaches the library itself.
"""
import os
import shutil
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

HEAD = r"""
import ctypes, sys
stub = ctypes.CDLL(sys.argv[1])
number = lambda name: ctypes.c_int.in_dll(stub, name)
sys.path.insert(0, sys.argv[2])
import torch
import stable_variance_amd as sv
dev = torch.device("cuda:0")
x, w, s = torch.ones(3, 8, device=dev), torch.ones(8, device=dev), torch.ones(3, device=dev)
calls = [lambda: sv.rms_norm(x, w), lambda: sv.rms_norm_fp8(x, w), lambda: sv.rms_norm_backward(x, x, s, w),
         lambda: sv.grad_norm([x]), lambda: sv.clip_grad_norm([x], 1.0), lambda: sv.clip_grad_norm([x], 1.0, out=[x])]
version = x._version
"""

FAILED = HEAD + r"""
number("stand_in_status").value = 4  # a launch failed
for i, call in enumerate(calls):
    try:
        call()
    except sv.SvError as e:
        assert e.status == 4
    else:
        raise AssertionError(f"call {i} was made again")
assert number("stand_in_calls").value == len(calls)
torch.cuda.synchronize()
assert (x == 1).all() and x._version == version
print("done")
"""

THREADS = HEAD + r"""
number("stand_in_status").value = 1  # refused: the general way makes the call
for call in calls:
    call()
torch.cuda.synchronize()
assert number("stand_in_calls").value == len(calls)
assert number("stand_in_with_gil").value == 0, number("stand_in_with_gil").value
print("done")
"""


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    so = str(tmp_path_factory.mktemp("stand_in") / "library_stand_in.so")
    res = subprocess.run([gcc, "-O1", "-Wall", "-Werror", "-shared", "-fPIC",
                          os.path.join(HERE, "library_stand_in.c"), "-o", so], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return so


def run(program, so):
    # before whatever else is preloaded here
    pre = " ".join(p for p in (so, os.environ.get("LD_PRELOAD", "")) if p)
    res = subprocess.run([sys.executable, "-c", program, so, os.path.dirname(HERE)], capture_output=True, text=True,
                         timeout=100, env={**os.environ, "LD_PRELOAD": pre})
    assert res.returncode == 0, res.stderr[-4000:]
    assert res.stdout.strip().splitlines()[-1] == "done"


def test_a_call_whose_launch_failed_is_not_made_again(stand_in):
    # some of it may have run: in place, a second one would scale twice
    run(FAILED, stand_in)


def test_other_threads_run_beside_the_library(stand_in):
    # a launch waits when the queue is full; a thread that the queue waits for
    # needs the interpreter's lock
    run(THREADS, stand_in)
