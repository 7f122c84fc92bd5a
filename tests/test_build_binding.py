"""Building the C++ form of the attention binding where something is missing, twice, or in several
processes: the library's build never fails for it, and a good module is never lost."""

import os
import sys
import types

import pytest
import torch

import memory_bound_decode_fd_gb300 as package
from memory_bound_decode_fd_gb300 import attention, build


@pytest.fixture
def module(monkeypatch, tmp_path):
    """A module of the present sources, built against another torch; a library that is up to date."""
    monkeypatch.setattr(build, "TORCH_PATH", tmp_path / "_fd_torch.so")
    monkeypatch.setattr(build, "TORCH_STAMP", tmp_path / "stamp")
    monkeypatch.setattr(build, "is_stale", lambda: False)
    build.TORCH_PATH.write_bytes(b"before")
    build.TORCH_STAMP.write_text("another torch")
    return build.TORCH_PATH


def older(path):
    os.utime(path, (0, 0))  # than its sources


def no_nvcc():
    raise RuntimeError("nvcc not found")


@pytest.mark.parametrize("why", ["no nvcc", "no headers", "no compiler"])
@pytest.mark.parametrize("current", [True, False])
def test_build_goes_on_without_it(module, monkeypatch, tmp_path, why, current):
    if why == "no nvcc":
        monkeypatch.setattr(build, "_nvcc", no_nvcc)
    elif why == "no headers":
        monkeypatch.setattr(build.sysconfig, "get_path", lambda name: str(tmp_path))
    else:
        monkeypatch.setenv("CXX", str(tmp_path / "none"))
    if not current:
        older(module)
    assert build.build() == build.LIB_PATH
    # a module of older sources would call the library by an older header
    assert module.exists() == current


def test_the_module_is_there_while_the_next_is_built(module, monkeypatch):
    seen = []

    def run(cmd, verbose):
        seen.append(module.read_bytes())
        open(cmd[cmd.index("-o") + 1], "wb").write(b"after")

    monkeypatch.setattr(build, "_run", run)
    build.build()
    assert seen == [b"before"] and module.read_bytes() == b"after"
    assert not build._torch_stale()


def test_processes_that_build_at_once_do_not_share_a_file(module, monkeypatch):
    names = []

    def run(cmd, verbose):
        out = cmd[cmd.index("-o") + 1]
        names.append(out)
        assert not os.path.exists(out)
        open(out, "wb").write(b"half")
        if len(names) == 1:  # another process builds meanwhile, and fails
            monkeypatch.setattr(build.os, "getpid", lambda: 1)
            build._build_torch(False)
            assert not os.path.exists(names[1])
            open(out, "ab").write(b"whole")
        else:
            raise RuntimeError("killed")

    monkeypatch.setattr(build, "_run", run)
    build._build_torch(False)
    assert names[0] != names[1] and module.read_bytes() == b"halfwhole"


def test_what_does_not_compile_is_not_tried_again(module, monkeypatch, tmp_path):
    runs = []

    def run(cmd, verbose):
        runs.append(cmd)
        raise RuntimeError("does not compile")

    monkeypatch.setattr(build, "_run", run)
    for _ in range(3):
        build.build()
    assert len(runs) == 1
    monkeypatch.setenv("CXX", "another")  # until there is another compiler,
    build.build()
    build.build()
    assert len(runs) == 2
    older(build.TORCH_STAMP)  # or another source
    build.build()
    build.build()
    assert len(runs) == 3
    # what is merely missing is looked for every time
    build.TORCH_STAMP.unlink()
    monkeypatch.setattr(build, "_nvcc", no_nvcc)
    build.build()
    assert build._torch_stale()


@pytest.mark.parametrize("torch_version,python_version,used", [
    (None, None, True), ("1.0", None, False), (None, "2.7", False), ("1.0", "2.7", False)])
def test_a_module_for_another_python_or_torch_is_not_used(fdlib, monkeypatch, torch_version, python_version, used):
    module = types.ModuleType("_fd_torch")
    module.torch_version = torch_version or torch.__version__
    module.python_version = python_version or f"{sys.version_info.major}.{sys.version_info.minor}"
    calls = []
    module.init = lambda *addresses: calls.append(addresses)
    monkeypatch.setattr(package, "_fd_torch", module, raising=False)
    monkeypatch.setitem(sys.modules, package.__name__ + "._fd_torch", module)
    monkeypatch.setattr(attention, "_fast", None)
    attention._load()
    assert attention._fast is (module if used else False)
    assert len(calls) == used  # nothing of it is called before it is known to fit


def test_the_module_names_the_python_it_is_for(fdlib):
    attention._load()
    if not attention._fast:
        pytest.skip("not built")
    assert attention._fast.python_version == f"{sys.version_info.major}.{sys.version_info.minor}"
