"""Build the CUDA library ``libdwc_gb300.so`` in-tree with nvcc, for sm_103a only.

Every ``csrc/*.cu`` file is compiled to an object in parallel, then linked into a shared
library next to this file.  Rebuilds only what changed (sources or headers newer than the
object).  No CPU fallback exists: importing the binding without this library fails loudly.

``csrc/dwc_norm_py.cpp``, the host path of the norm operators for Python, is compiled beside it with
the host compiler against the installed PyTorch and linked as the module ``_norm_host``.  Run as a
script (``python depthwise_convolution_nhwc_gb300/_build.py``) where there is no PyTorch, the build makes the C
library alone.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libdwc_gb300.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
HOST_SRC = os.path.join(CSRC, "dwc_norm_py.cpp")
HOST_PATH = os.path.join(HERE, "_norm_host.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdwc_gb300.so")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _stale(obj: str, src: str, hdr_mtime: float) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return t < os.path.getmtime(src) or t < hdr_mtime


def _host_object() -> str | None:
    """The host module's object file, one per PyTorch and Python version; none without PyTorch."""
    try:
        import torch
    except ImportError:
        return None
    return os.path.join(OBJ_DIR, f"dwc_norm_py-{torch.__version__}-{sys.version_info[0]}{sys.version_info[1]}.o")


def _compile_host(obj: str) -> None:
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
            os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")]
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    tmp = obj + f".tmp{os.getpid()}"
    r = subprocess.run(cmd + [f"-I{d}" for d in dirs] + ["-c", HOST_SRC, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {os.path.basename(HOST_SRC)}:\n{r.stderr[-6000:]}")
    os.replace(tmp, obj)


def _host_linked(obj: str) -> bool:
    """Whether the host module was linked from this object as it is now (objects of several PyTorch
    versions share one module; which of them it holds is recorded beside them)."""
    try:
        with open(_host_record()) as f:
            return f.read() == os.path.basename(obj) and os.path.getmtime(HOST_PATH) >= os.path.getmtime(obj)
    except OSError:
        return False


def _host_record() -> str:
    return os.path.join(OBJ_DIR, "dwc_norm_py.linked")


def _link_host(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = HOST_PATH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-shared", "-o", tmp, obj, "-L", HERE,
           f"-l:{LIB_NAME}", "-L", lib, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(HOST_PATH)} failed:\n{r.stderr[-6000:]}")
    os.replace(tmp, HOST_PATH)


def build(verbose: bool = False, jobs: int | None = None, extra_flags=None) -> str:
    """Compile and link the library; returns its path."""
    nvcc = nvcc_path()
    os.makedirs(OBJ_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_mtime = max((os.path.getmtime(h) for h in _headers()), default=0.0)
    objs = [os.path.join(OBJ_DIR, os.path.basename(s)[:-3] + ".o") for s in srcs]
    flags = NVCC_FLAGS + list(extra_flags or [])
    if verbose:
        flags = flags + ["-Xptxas", "-v"]

    todo = [(s, o) for s, o in zip(srcs, objs) if _stale(o, s, hdr_mtime)]

    def compile_one(so):
        s, o = so
        cmd = [nvcc] + ARCH + flags + ["-c", s, "-o", o + ".tmp"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(s)}:\n{r.stderr[-6000:]}")
        os.replace(o + ".tmp", o)
        return s, r.stderr

    host_obj = _host_object()
    host_todo = host_obj is not None and _stale(host_obj, HOST_SRC, hdr_mtime)
    jobs = jobs or min(len(todo) + host_todo, os.cpu_count() or 4) or 1
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        host = ex.submit(_compile_host, host_obj) if host_todo else None
        for s, log in ex.map(compile_one, todo):
            if verbose and log:
                sys.stderr.write(f"== {os.path.basename(s)}\n{log}")
        if host is not None:
            host.result()

    if todo or not os.path.exists(LIB_PATH):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr[-6000:]}")
        os.replace(tmp, LIB_PATH)
    if host_obj is not None and not _host_linked(host_obj):
        _link_host(host_obj)
        with open(_host_record(), "w") as f:
            f.write(os.path.basename(host_obj))
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
