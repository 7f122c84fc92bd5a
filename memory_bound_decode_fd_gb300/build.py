"""Build ``libfd.so`` (the C-ABI CUDA library) in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` is compiled to an object in parallel, then linked into one shared
library next to this file. The CUDA runtime is linked statically, so the library needs
only the NVIDIA driver at run time. ``build()`` is a no-op when the library is newer
than every source and header.

``csrc/fd_torch.cpp`` becomes ``_fd_torch.so``, the C++ form of attention.py's calls, against
the headers of the torch that is installed. Where those or Python's are missing it is left out,
and the calls do the same in Python.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
from pathlib import Path

PKG_DIR = Path(__file__).resolve().parent
REPO_DIR = PKG_DIR.parent
CSRC = PKG_DIR / "csrc"
INCLUDE = REPO_DIR / "include"
BUILD_DIR = REPO_DIR / "_build"
LIB_PATH = PKG_DIR / "libfd.so"
TORCH_SRC = CSRC / "fd_torch.cpp"
TORCH_PATH = PKG_DIR / "_fd_torch.so"
TORCH_STAMP = BUILD_DIR / "fd_torch.torch"  # the torch that TORCH_PATH was built against

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", f"-I{INCLUDE}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found: the fd CUDA library cannot be built")


def _sources() -> list[Path]:
    return sorted(CSRC.glob("*.cu"))


def _deps() -> list[Path]:
    return _sources() + sorted(CSRC.glob("*.h")) + sorted(CSRC.glob("*.cuh")) + sorted(
        INCLUDE.glob("*.h")
    ) + [Path(__file__)]


def is_stale() -> bool:
    if not LIB_PATH.exists():
        return True
    lib_mtime = LIB_PATH.stat().st_mtime
    return any(p.stat().st_mtime > lib_mtime for p in _deps())


def _torch_version() -> str | None:
    try:
        import torch
    except ImportError:
        return None
    return f"{torch.__version__} {sys.version}"


def _torch_older(path: Path) -> bool:
    """Whether ``path`` is older than what ``_fd_torch.so`` is made from."""
    made = path.stat().st_mtime
    return any(p.stat().st_mtime > made for p in (TORCH_SRC, INCLUDE / "fd.h"))


def _cxx() -> str:
    return os.environ.get("CXX", "g++")


def _not_built() -> str:
    """What TORCH_STAMP holds where ``_fd_torch.so`` does not compile."""
    return f"{_torch_version()} not built with {_cxx()}"


def _torch_stale() -> bool:
    stamp = TORCH_STAMP.read_text() if TORCH_STAMP.exists() else None
    if stamp == _not_built():
        return _torch_older(TORCH_STAMP)
    return stamp != _torch_version() or not TORCH_PATH.exists() or _torch_older(TORCH_PATH)


def _build_torch(verbose: bool) -> None:
    """``_fd_torch.so``. Where it cannot be built, one from before is left if it is of the present
    sources (that it is of another torch is found when it is loaded), else removed."""

    def leave_out(why: Exception | None = None) -> None:
        if TORCH_PATH.exists() and _torch_older(TORCH_PATH):
            TORCH_PATH.unlink(missing_ok=True)
        if why:
            print(f"_fd_torch.so not built, attention.py's calls stay in Python: {why}", file=sys.stderr)

    version, python = _torch_version(), sysconfig.get_path("include")
    if version is None or not Path(python, "Python.h").exists():
        return leave_out()
    import torch

    root = Path(torch.__file__).parent
    tmp = TORCH_PATH.with_name(f"_fd_torch.{os.getpid()}.tmp.so")  # of this process: others may build too
    try:
        cuda = Path(_nvcc()).resolve().parent.parent
    except RuntimeError as e:
        return leave_out(e)
    try:
        _run([_cxx(), "-O2", "-std=c++17", "-fPIC", "-shared", f"-I{INCLUDE}",
              f"-I{root / 'include'}", f"-I{root / 'include/torch/csrc/api/include'}", f"-I{python}",
              f"-I{cuda / 'include'}", f'-DFD_TORCH_VERSION="{torch.__version__}"',
              f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", str(TORCH_SRC), "-o", str(tmp),
              f"-L{root / 'lib'}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"], verbose)
    except (RuntimeError, OSError) as e:
        tmp.unlink(missing_ok=True)
        if isinstance(e, RuntimeError):  # it does not compile: not tried again until something is new
            TORCH_STAMP.write_text(_not_built())
        return leave_out(e)
    os.replace(tmp, TORCH_PATH)
    TORCH_STAMP.write_text(version)


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(
            f"command failed ({proc.returncode}): {' '.join(cmd)}\n{proc.stdout}\n{proc.stderr}"
        )
    if verbose and (proc.stdout or proc.stderr):
        print(proc.stdout + proc.stderr, flush=True)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> Path:
    """Compile and link ``libfd.so``; return its path."""
    BUILD_DIR.mkdir(exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        beside = ex.submit(_build_torch, verbose) if force or _torch_stale() else None
        if force or is_stale():
            _build_lib(verbose, ptxas_info)
        if beside:
            beside.result()
    return LIB_PATH


def _build_lib(verbose: bool, ptxas_info: bool) -> None:
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    jobs = []
    for src in _sources():
        obj = BUILD_DIR / (src.stem + ".o")
        jobs.append((obj, [nvcc, *ARCH_FLAGS, *COMMON_FLAGS, *extra, "-c", str(src), "-o", str(obj)]))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        list(ex.map(lambda j: _run(j[1], verbose or ptxas_info), jobs))
    tmp = LIB_PATH.with_suffix(".so.tmp")
    _run([nvcc, *ARCH_FLAGS, "-shared", "-o", str(tmp), *[str(o) for o, _ in jobs]], verbose)
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
