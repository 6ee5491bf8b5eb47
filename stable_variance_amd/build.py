"""Build libstable_variance.so for gfx950 with hipcc, and the module sv_torch
that passes torch's tensors to it, with g++ (both in-tree, no JIT cache)."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "sv_lib.hip")
# In this order the build guards' search over all assembly is short: they look
# for every kernel from its start, so many small kernels come first.
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


def module_tag() -> str:
    """What the module is made for, as its file says it."""
    import torch

    return f"sv_torch for torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"


def module_fits(path: str = None) -> bool:
    """Whether a built module is made for the torch and the Python that run."""
    with open(path or MODULE, "rb") as f:
        return module_tag().encode() + b"\0" in f.read()


def module_commands(obj: str, out: str):
    """The compile and the link command of the module; the link needs LIB."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    dirs = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
            os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(hipcc()))), "include"),
            sysconfig.get_paths()["include"]]
    cxx = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DSV_TORCH_TAG="{module_tag()}"']
    for d in dirs:
        cxx += ["-isystem", d]
    link = ["g++", "-shared", obj, "-L" + OUT_DIR, "-l:" + os.path.basename(LIB), "-L" + os.path.join(root, "lib"),
            "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-o", out]
    return [*cxx, "-c", MODULE_SRC, "-o", obj], link


def _start(cmd):
    try:
        return cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
    except OSError as e:  # no such compiler
        return cmd, e


def _failure(cmd, started, verbose: bool) -> str:
    """Waits for a command: what it said if it failed, else nothing."""
    if isinstance(started, Exception):
        return f"{' '.join(cmd)}\n{started}\n"
    out, err = started.communicate()
    if started.returncode != 0:
        return " ".join(cmd) + "\n" + out + err
    if verbose:
        print(" ".join(cmd))
    return ""


def has_torch() -> bool:
    """Whether torch is installed here: the module needs it, the library does not."""
    return importlib.util.find_spec("torch") is not None


def build(verbose: bool = False) -> str:
    """Compile the sources (in parallel) and link the library and, where torch
    is installed, the module; returns the library's path.  The library needs
    hipcc alone and is in place before a failure of the module is raised."""
    os.makedirs(OUT_DIR, exist_ok=True)
    module_obj, module_tmp = os.path.join(OUT_DIR, "sv_torch.o"), MODULE + ".tmp"
    module, link_module = None, None
    if has_torch():
        try:
            compile_module, link_module = module_commands(module_obj, module_tmp)
            module = _start(compile_module)
        except ImportError as e:
            module = ["import torch"], e
    flags = [f for f in HIPCC_FLAGS if f != "-shared"]
    objs, started = [], []
    for src in SRCS:
        obj = os.path.join(OUT_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        started.append(_start([hipcc(), *flags, "-c", src, "-o", obj]))
        objs.append(obj)
    errors = [e for e in [_failure(*s, verbose) for s in started] if e]
    module_error = _failure(*module, verbose) if module else ""
    if errors:
        raise RuntimeError("hipcc failed:\n" + "\n".join(errors))
    tmp = LIB + ".tmp"
    error = _failure(*_start([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]), verbose)
    if error:
        raise RuntimeError("link failed:\n" + error)
    os.replace(tmp, LIB)
    for obj in objs:
        os.remove(obj)
    if module:
        module_error = module_error or _failure(*_start(link_module), verbose)
        if module_error:
            raise RuntimeError(f"{LIB} is built, the module sv_torch is not:\n" + module_error)
        os.replace(module_tmp, MODULE)
        os.remove(module_obj)
    return LIB


def is_stale() -> bool:
    built, sources = [LIB], DEPS
    if has_torch():
        built, sources = [LIB, MODULE], [*DEPS, MODULE_SRC]
    if not all(map(os.path.exists, built)) or (MODULE in built and not module_fits()):
        return True
    t = min(map(os.path.getmtime, built))
    return any(os.path.getmtime(d) > t for d in sources)


if __name__ == "__main__":
    print(build(verbose=True))
