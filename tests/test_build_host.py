"""The C++ form of the attention binding: built with the library, against the installed torch, and
left out without harm where it cannot be."""

import sysconfig
from pathlib import Path

import pytest
import torch

from memory_bound_decode_fd_gb300 import attention, build


def test_built_against_this_torch(fdlib):
    if not Path(sysconfig.get_path("include"), "Python.h").exists():
        pytest.skip("no Python headers")
    attention._load()
    assert attention._fast and attention._fast.torch_version == torch.__version__
    assert not build._torch_stale()


def test_arguments_it_does_not_take_come_back(fdlib):
    attention._load()
    if not attention._fast:
        pytest.skip("not built")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    f, pos = torch.ones(32, dtype=torch.float64), torch.zeros(2, dtype=torch.int32)
    fast = attention._fast
    assert fast.rope(q, None, pos, f, False, 1.0, None, None) is None  # on the CPU
    for bad in ((), (q,), (1, 2, 3, 4, 5, 6, 7, 8), (None,) * 8, (q, None, pos, f, 0, "x", None, None)):
        assert fast.rope(*bad) is None
    for n in (0, 1, 12, 13, 14, 15):
        assert fast.rope_append(*(None,) * n) is None and fast.paged_attention(*(None,) * n) is None
        assert fast.rope_append(*(q,) * n) is None and fast.paged_attention(*(q,) * n) is None
    with pytest.raises(TypeError):
        fast.init(1)


@pytest.mark.parametrize("why", ["no headers", "no compiler", "does not compile"])
def test_left_out_where_it_cannot_be_built(monkeypatch, tmp_path, capsys, why):
    monkeypatch.setattr(build, "TORCH_PATH", tmp_path / "_fd_torch.so")
    monkeypatch.setattr(build, "TORCH_STAMP", tmp_path / "stamp")
    if why == "no headers":
        monkeypatch.setattr(build.sysconfig, "get_path", lambda name: str(tmp_path))
    elif why == "no compiler":
        monkeypatch.setenv("CXX", str(tmp_path / "none"))
    else:
        bad = tmp_path / "fd_torch.cpp"
        bad.write_text("#error no\n")
        monkeypatch.setattr(build, "TORCH_SRC", bad)
    build._build_torch(False)
    assert not build.TORCH_PATH.exists()
    assert (capsys.readouterr().err == "") == (why == "no headers")
