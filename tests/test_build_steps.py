"""The build's steps with stand-ins for the compilers: the library needs hipcc
alone, the module that takes torch's tensors to it torch and g++ too."""
import os
import sys
import warnings

import pytest
import torch

import stable_variance_amd as sv
from stable_variance_amd import build as libbuild

WORKS = """#!/bin/sh
while [ $# -gt 0 ]; do
  if [ "$1" = -o ]; then printf '%s\\0' "$MADE_FOR" > "$2"; fi
  shift
done
"""
FAILS = "#!/bin/sh\necho it does not compile >&2\nexit 1\n"


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """tools(hipcc, g++): the scripts that stand in for them (None: there is
    none); libraries go to a folder of their own."""
    out, tools = tmp_path / "lib", tmp_path / "tools"
    tools.mkdir()
    monkeypatch.setattr(libbuild, "OUT_DIR", str(out))
    monkeypatch.setattr(libbuild, "LIB", str(out / "libstable_variance.so"))
    monkeypatch.setattr(libbuild, "MODULE", str(out / "sv_torch.so"))
    monkeypatch.setenv("MADE_FOR", libbuild.module_tag())

    def use(hipcc, gxx):
        for name, script in (("hipcc", hipcc), ("g++", gxx)):
            if script is not None:
                (tools / name).write_text(script)
                (tools / name).chmod(0o755)
        # the scripts take the shell's own commands only, so that no compiler of
        # the system's is found
        monkeypatch.setenv("PATH", str(tools))
        monkeypatch.setattr(libbuild, "hipcc", lambda: str(tools / "hipcc"))

    return use


def left():
    return sorted(os.listdir(libbuild.OUT_DIR))


def test_both(tools):
    tools(WORKS, WORKS)
    assert libbuild.build() == libbuild.LIB
    assert left() == ["libstable_variance.so", "sv_torch.so"] and not libbuild.is_stale()
    os.remove(libbuild.MODULE)
    assert libbuild.is_stale()


@pytest.mark.parametrize("version", ["2.9.1", torch.__version__ + "1", torch.__version__[:-1]])
def test_a_module_for_another_torch_is_stale(tools, monkeypatch, version):
    tools(WORKS, WORKS)
    monkeypatch.setenv("MADE_FOR", libbuild.module_tag().replace(torch.__version__, version))
    libbuild.build()
    assert libbuild.is_stale()
    monkeypatch.setattr(sv, "_native", None)
    monkeypatch.setattr(sv, "_MODULE_PATH", libbuild.MODULE)
    with pytest.raises(ImportError, match="is not sv_torch for torch"):
        sv.native()  # and not the loader's error, or a crash


def test_the_module_says_what_it_is_made_for():
    assert libbuild.module_fits()
    assert sv.native().__doc__ == libbuild.module_tag()


@pytest.mark.parametrize("gxx", [WORKS, FAILS, None], ids=["works", "fails", "none"])
def test_the_library_is_built_without_torch(tools, monkeypatch, gxx):
    tools(WORKS, gxx)
    monkeypatch.setitem(sys.modules, "torch", None)  # as if it was not installed
    assert libbuild.build() == libbuild.LIB
    assert left() == ["libstable_variance.so"] and not libbuild.is_stale()


@pytest.mark.parametrize("gxx", [FAILS, None], ids=["fails", "none"])
def test_the_library_is_built_where_the_module_is_not(tools, gxx):
    tools(WORKS, gxx)
    with pytest.raises(RuntimeError, match="sv_torch"):
        libbuild.build()
    assert "libstable_variance.so" in left() and "sv_torch.so" not in left()
    assert libbuild.is_stale()


def test_the_library_is_built_beside_a_torch_that_does_not_load(tools, monkeypatch):
    def broken(*_):
        raise ImportError("libtorch.so: no such file")

    tools(WORKS, WORKS)
    monkeypatch.setattr(libbuild, "module_commands", broken)
    with pytest.raises(RuntimeError, match="libtorch"):
        libbuild.build()
    assert left() == ["libstable_variance.so"]


@pytest.mark.parametrize("hipcc", [FAILS, None], ids=["fails", "none"])
def test_no_module_without_the_library(tools, hipcc):
    tools(hipcc, WORKS)
    with pytest.raises(RuntimeError, match="hipcc"):
        libbuild.build()
    assert not any(name.endswith(".so") for name in left())


def test_the_calls_need_the_library_alone(tools, monkeypatch):
    # the module absent or for another torch: said once, and the calls go on
    tools(WORKS, WORKS)
    monkeypatch.setenv("MADE_FOR", "another")
    libbuild.build()
    x, s = torch.zeros(3, 4), torch.zeros(3)
    for path in (libbuild.MODULE, libbuild.MODULE + ".none"):
        monkeypatch.setattr(sv, "_native", None)
        monkeypatch.setattr(sv, "_short_way", None)
        monkeypatch.setattr(sv, "_MODULE_PATH", path)
        with pytest.warns(RuntimeWarning, match="longer way"), pytest.raises(ValueError):
            sv.rms_norm(x)
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            for call in (lambda: sv.rms_norm(x), lambda: sv.rms_norm_fp8(x), lambda: sv.grad_norm([x]),
                         lambda: sv.rms_norm_backward(x, x, s, x[0]), lambda: sv.clip_grad_norm([x], 1.0)):
                with pytest.raises(ValueError):  # not on a HIP device: the general way has looked at it
                    call()
    monkeypatch.setattr(sv, "_short_way", None)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(RuntimeWarning):
            sv.rms_norm(x)
        with pytest.raises(ValueError):  # also where the warning is made an error
            sv.rms_norm(x)
    monkeypatch.setattr(sv, "_short_way", None)
    monkeypatch.setattr(sv, "_lib", None)
    monkeypatch.setattr(sv, "_LIB_PATH", libbuild.LIB + ".none")
    with pytest.raises(ImportError, match="libstable_variance"):
        sv.rms_norm(x)
