"""Build the in-tree shared library ``libmla_lowbit.so`` with nvcc for sm_103a.

One nvcc invocation compiles every ``csrc/*.cu`` file (in parallel with
``--threads``) and links them into ``bit_mla_kv_lowbit_gb300/libmla_lowbit.so``.
The build is skipped when the library is newer than every source and header.

Beside it, ``csrc/marshal.cpp`` becomes a small Python extension (the argument
checks and the launch of the serving-step calls), compiled with g++ against the
installed torch and named after its version.  Where that cannot be built the
binding does the same in Python.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmla_lowbit.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; set NVCC or put the CUDA toolkit on PATH")


MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")


def marshal_path() -> str:
    """The argument-marshalling extension for the installed torch."""
    from importlib import metadata
    tag = metadata.version("torch").replace("+", "_").replace(".", "_")
    return os.path.join(PKG, f"_marshal_torch{tag}_py{sys.version_info[0]}{sys.version_info[1]}.so")


def _start_marshal(force: bool):
    """Start compiling the extension; ``(process, temporary, target)`` or None
    when it is up to date or cannot be built here."""
    try:
        import sysconfig
        from importlib import util
        target = marshal_path()
        newest = max(map(os.path.getmtime, [MARSHAL_SRC, os.path.abspath(__file__), *glob.glob(os.path.join(INCLUDE, "*.h"))]))
        if not force and os.path.exists(target) and os.path.getmtime(target) >= newest:
            return None
        torch_dir = os.path.dirname(util.find_spec("torch").origin)
        gxx = shutil.which("g++")
        if gxx is None:
            return None
        tmp = target + ".tmp"
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
        cmd = [gxx, "-std=c++17", "-O2", "-fPIC", "-shared", f"-I{torch_dir}/include",
               f"-I{torch_dir}/include/torch/csrc/api/include", f"-I{sysconfig.get_paths()['include']}",
               f"-I{cuda}/include", f"-I{INCLUDE}", MARSHAL_SRC, "-o", tmp, f"-L{torch_dir}/lib", "-ltorch_python",
               "-ltorch_cpu", "-lc10", "-lc10_cuda"]
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True), tmp, target
    except Exception as e:  # no torch, no headers: the binding's own checks serve
        sys.stderr.write(f"the argument-marshalling extension is not built: {e}\n")
        return None


def _finish_marshal(job) -> None:
    if job is None:
        return
    proc, tmp, target = job
    log, _ = proc.communicate()
    if proc.returncode == 0:
        os.replace(tmp, target)
    else:
        sys.stderr.write(f"the argument-marshalling extension is not built:\n{log[-2000:]}\n")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + [h for d, e in ((CSRC, "cuh"), (CSRC, "h"), (INCLUDE, "h")) for h in glob.glob(os.path.join(d, f"*.{e}"))]
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps)


def build_library(force: bool = False, verbose: bool = False) -> str:
    job = _start_marshal(force)
    try:
        return _build_lib(force, verbose)
    finally:
        _finish_marshal(job)


def _build_lib(force: bool, verbose: bool) -> str:
    if not force and not _stale():
        return LIB
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "--threads", "0",
           "-Xcompiler", "-fPIC", "-shared", f"-I{INCLUDE}", "-o", tmp, *sources(),
           "-lcudart"]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed building libmla_lowbit.so")
    if verbose:
        sys.stderr.write(res.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
