"""Build the CUDA library libmla_decode.so in-tree with nvcc (sm_103a only), and
beside it _mla_host.<tag>.so, the argument marshalling of the tree step's calls
on torch's tensor objects (host C++, against the installed torch's headers; the
tag names the Python ABI and the torch that it fits, and no other loads it).

The library needs neither torch nor Python's headers.  Where the host module cannot
be built, a warning says why and the binding marshals those calls in Python.

All translation units compile in parallel and link with -shared; the CUDA
runtime links statically and the driver API is reached through
cudaGetDriverEntryPoint.  At load time the library needs nothing but libc and
the NVIDIA driver: every kernel is this library's own.
"""

from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libmla_decode.so")
HOST_SRC = os.path.join(CSRC, "host", "mla_host.cpp")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmla_decode.so")


def host_path() -> str:
    """The host module that fits this Python and the installed torch (both lay out what it reads)."""
    import sysconfig

    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(HERE, f"_mla_host.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}-{abi}.so")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return files + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]


def _newer(built: str, files: list[str]) -> bool:
    return os.path.exists(built) and all(os.path.getmtime(f) <= os.path.getmtime(built) for f in files)


def _library_up_to_date() -> bool:
    return _newer(LIB_PATH, sources() + _headers())


def _host_up_to_date() -> bool:
    if importlib.util.find_spec("torch") is None:
        return True
    try:
        path = host_path()
    except Exception:   # a torch that does not import: building says why
        return False
    return _newer(path, [HOST_SRC] + _headers())


def up_to_date() -> bool:
    return _library_up_to_date() and _host_up_to_date()


def _build_host() -> None:
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    inc = [INCLUDE, os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], cuda]
    path = host_path()
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[x for d in inc for x in ("-isystem" if d != INCLUDE else "-I", d)], HOST_SRC, "-o", tmp,
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {HOST_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def _build_library(ex: cf.Executor, verbose: bool, extra_flags: tuple) -> None:
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    common = [nvcc, ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-I", INCLUDE, *extra_flags]
    if verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [*common, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    objs = list(ex.map(compile_one, sources()))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


def build(force: bool = False, verbose: bool = False, extra_flags: tuple = ()) -> str:
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        torch_here = importlib.util.find_spec("torch") is not None
        host = ex.submit(_build_host) if torch_here and (force or not _host_up_to_date()) else None
        if force or not _library_up_to_date():
            _build_library(ex, verbose, extra_flags)
        if host is not None:
            try:
                host.result()
            except Exception as e:
                warnings.warn(f"the host module was not built (calls are marshalled in Python): {e}", stacklevel=2)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
