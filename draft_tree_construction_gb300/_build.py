"""Compile the CUDA library (libdarttree.so) in-tree for sm_103a with nvcc.

Each translation unit compiles in parallel, then one nvcc call links the
shared library next to this file.  Objects go to ``_build/`` (git-ignored).
The Python module _steps_native (host C++ against PyTorch's headers, no device
code) is compiled beside them, with the host compiler; the library is linked
whether or not that succeeds.
"""
from __future__ import annotations

import contextlib
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdarttree.so")
NATIVE_SOURCE = os.path.join(CSRC, "dart_steps_py.cpp")
SOURCES = ["dart_api.cu", "dart_rows.cu", "dart_tree.cu", "dart_select.cu", "dart_probe.cu",
           "dart_adjust.cu", "dart_append.cu", "dart_attend.cu"]

NVCC = os.environ.get("NVCC", "nvcc")
CXX = os.environ.get("CXX", "g++")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files.append(os.path.join(INCLUDE, "darttree.h"))
    return files


def _native_inputs():
    return [NATIVE_SOURCE, os.path.join(INCLUDE, "darttree.h")]


def native_path() -> str | None:
    """The module's file for this interpreter and this PyTorch, whose binary interfaces it is bound to (None without
    PyTorch)."""
    try:
        import torch
    except ImportError:
        return None
    tag = f"torch-{torch.__version__}-{(torch.version.git_version or '')[:8]}"
    return os.path.join(HERE, f"_steps_native.{tag}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _modules() -> list[str]:
    """The modules of every PyTorch that the tree was built with: those of an older library go with it, whose
    structures may lie differently."""
    return glob.glob(os.path.join(glob.escape(os.path.dirname(LIB)), "_steps_native.*.so"))


def _stale(target: str, inputs: list[str]) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(f) > os.path.getmtime(target) for f in inputs)


def _native_stale() -> bool:
    path = native_path()
    return path is not None and _stale(path, _native_inputs())


def needs_build() -> bool:
    return _stale(LIB, _inputs()) or (_native_stale() and not _native_failed)


def _native_command(target: str) -> list[str]:
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(NVCC) or "/usr/local/cuda/bin/nvcc")))
    return [CXX, "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            "-I", INCLUDE, "-isystem", os.path.join(home, "include"),
            "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"], NATIVE_SOURCE,
            "-o", target, "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            f"-Wl,-rpath,{os.path.join(home, 'lib')}"]


# The library needs nvcc alone; the Python module also PyTorch's headers, and the
# steps work without it.  So a module that cannot be built is said so once a
# process and does not keep the library from being linked.
_native_failed = False


def _start_native(target: str):
    """(the module's running compilation, "") or (None, why there is none)."""
    try:
        return subprocess.Popen(_native_command(target), stdout=subprocess.PIPE, stderr=subprocess.STDOUT), ""
    except Exception as e:                 # no PyTorch, no host compiler
        return None, f"{type(e).__name__}: {e}"


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    global _native_failed
    want_lib = force or _stale(LIB, _inputs())
    path, why = native_path(), ""
    want_native = path is not None and (force or (_native_stale() and not _native_failed))
    native = f"{path}.{os.getpid()}.tmp"
    compiling = None
    if want_native:
        compiling, why = _start_native(native)
    try:
        if want_lib:
            _build_library(verbose, list(extra_flags or []))
            for old in _modules():
                if old != path:
                    os.remove(old)
    except BaseException:
        _finish_native(compiling)
        _remove(native)
        raise
    if want_native:
        why = why or _finish_native(compiling)
        _native_failed = bool(why)
        if why:
            _remove(native)
            _remove(path)                      # of other sources: its structures may lie differently
            warnings.warn(f"_steps_native was not built, calls of the steps around a tree take some microseconds "
                          f"longer:\n{why}", RuntimeWarning, stacklevel=2)
        else:
            os.replace(native, path)
    return LIB


def _finish_native(compiling) -> str:
    """What went wrong with the compilation, "" if nothing did."""
    if compiling is None:
        return ""
    out, _ = compiling.communicate()
    if compiling.returncode == 0:
        return ""
    return out.decode(errors="replace") or f"the host compiler returned {compiling.returncode}"


def _remove(path: str) -> None:
    with contextlib.suppress(FileNotFoundError):
        os.remove(path)


def _build_library(verbose: bool, extra: list[str]) -> None:
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if failed:
        msg = "\n".join(f"--- {s}\n{o}" for s, o in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    tmp = LIB + ".tmp"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
