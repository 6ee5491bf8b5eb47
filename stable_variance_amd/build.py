"""Build libstable_variance.so for gfx950 with hipcc, and the module sv_torch
that passes torch's tensors to it, with g++ (both in-tree, no JIT cache)."""
from __future__ import annotations

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "sv_lib.hip")
SRCS = [os.path.join(HERE, "csrc", name) for name in (
    "sv_gnorm.hip", "sv_f64.hip", "sv_rms.hip", "sv_rms_grad.hip", "sv_embed.hip", "sv_lib.hip", "sv_norm.hip",
    "sv_rms_fp8.hip", "sv_adn.hip", "sv_adn_folds_9_14.hip", "sv_adn_folds_15_21.hip")]
DEPS = SRCS + [os.path.join(HERE, "csrc", "sv_device.hpp"), os.path.join(HERE, "csrc", "sv_host.hpp"),
               os.path.join(HERE, "csrc", "sv_index.hpp"), os.path.join(HERE, "csrc", "sv_adn_kernel.hpp"),
               os.path.join(HERE, "csrc", "sv_rows.hpp"), os.path.join(HERE, "csrc", "sv_rms.hpp"),
               os.path.join(HERE, "csrc", "sv_rms_rows.hpp"),
               os.path.join(ROOT, "include", "stable_variance.h")]
MODULE_SRC = os.path.join(HERE, "csrc", "sv_torch.cpp")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libstable_variance.so")
MODULE = os.path.join(OUT_DIR, "sv_torch.so")

# -ffp-contract=off and no fast-math keep every TwoSum operation rounded on
# its own; packed FP32 instructions are disabled for the device code.
HIPCC_FLAGS = [
    "-O3", "--offload-arch=gfx950", "-std=c++17", "-fPIC", "-shared",
    "-ffp-contract=off", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wextra",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "hipcc"


def module_commands(obj: str, out: str):
    """The compile and the link command of the module; the link needs LIB."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    dirs = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
            os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(hipcc()))), "include"),
            sysconfig.get_paths()["include"]]
    cxx = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in dirs:
        cxx += ["-isystem", d]
    link = ["g++", "-shared", obj, "-L" + OUT_DIR, "-l:" + os.path.basename(LIB), "-L" + os.path.join(root, "lib"),
            "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-o", out]
    return [*cxx, "-c", MODULE_SRC, "-o", obj], link


def build(verbose: bool = False) -> str:
    """Compile the sources (in parallel) and link the library and the module; returns the library's path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    flags = [f for f in HIPCC_FLAGS if f != "-shared"]
    module_obj, module_tmp = os.path.join(OUT_DIR, "sv_torch.o"), MODULE + ".tmp"
    compile_module, link_module = module_commands(module_obj, module_tmp)
    objs = []
    procs = [(compile_module, subprocess.Popen(compile_module, stdout=subprocess.PIPE, stderr=subprocess.PIPE,
                                               text=True))]
    for src in SRCS:
        obj = os.path.join(OUT_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [hipcc(), *flags, "-c", src, "-o", obj]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
        objs.append(obj)
    errors = []
    for cmd, pr in procs:
        out, err = pr.communicate()
        if pr.returncode != 0:
            errors.append(" ".join(cmd) + "\n" + out + err)
        elif verbose:
            print(" ".join(cmd))
    if errors:
        raise RuntimeError("hipcc failed:\n" + "\n".join(errors))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    if verbose:
        print(" ".join(cmd))
    os.replace(tmp, LIB)
    res = subprocess.run(link_module, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n" + " ".join(link_module) + "\n" + res.stdout + res.stderr)
    if verbose:
        print(" ".join(link_module))
    os.replace(module_tmp, MODULE)
    for obj in [*objs, module_obj]:
        os.remove(obj)
    return LIB


def is_stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MODULE):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(MODULE))
    return any(os.path.getmtime(d) > t for d in [*DEPS, MODULE_SRC])


if __name__ == "__main__":
    print(build(verbose=True))
