"""Build ``libpa_b200.so`` in-tree: the sm_100a kernels, the C ABI and the host
block manager, compiled with nvcc for ``-gencode arch=compute_100a,code=sm_100a``;
and ``_step.so``, the compiled binding of the serving-step calls (against torch's headers).

``python paged_kv_cache_389_b200/build.py [--force]`` (run as a script: importing the
package needs the built library).  nvcc cross-compiles, so
this runs without a GPU.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
CSRC = os.path.join(PKG, "csrc")
HOST = os.path.join(PKG, "host")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpa_b200.so")
BINDING = os.path.join(PKG, "binding", "step.cpp")
STEP = os.path.join(PKG, "_step.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CUDA_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler",
                     "-fvisibility=hidden", "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]
HOST_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-Wextra", "-I", INCLUDE]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu"))) + sorted(glob.glob(os.path.join(HOST, "*.cpp")))


def headers():
    return (glob.glob(os.path.join(INCLUDE, "*.h")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(CSRC, "*.cuh")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in sources() + headers() + [__file__])


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    if src.endswith(".cu"):
        cmd = [NVCC] + CUDA_FLAGS + extra + ["-c", src, "-o", obj]
    else:
        cmd = ["g++"] + HOST_FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _made_for() -> str | None:
    """What the binding is compiled against: Python and torch.  None where there is no torch."""
    if importlib.util.find_spec("torch") is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        import torch
        version = torch.__version__
    return f"{sys.implementation.cache_tag} torch {version}"


def build_binding(force: bool = False) -> str | None:
    """Compile the binding of the serving-step calls, linked to the library beside it.  It is
    compiled again when its source, Python or torch has changed.  Without torch (or with one
    without CUDA) there is nothing that could call it: the library is built alone, and None returned."""
    made_for, stamp = _made_for(), os.path.join(OBJ, "step.made_for")
    if made_for is None:
        print("no torch: the binding of the serving-step calls is left out", file=sys.stderr)
        return None
    inputs = [BINDING, os.path.join(INCLUDE, "pa.h"), __file__]
    if not force and os.path.exists(STEP) and all(os.path.getmtime(f) <= os.path.getmtime(STEP) for f in inputs):
        if os.path.exists(stamp) and open(stamp).read() == made_for:
            return STEP
    import sysconfig
    import torch
    from torch.utils import cpp_extension
    if torch.version.cuda is None:
        print("torch without CUDA: the binding of the serving-step calls is left out", file=sys.stderr)
        return None
    os.makedirs(OBJ, exist_ok=True)
    tmp = STEP + f".tmp{os.getpid()}"
    dirs = [INCLUDE] + cpp_extension.include_paths() + [os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
                                                        sysconfig.get_paths()["include"]]
    libs = cpp_extension.library_paths()
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", BINDING, "-o", tmp, "-I" + dirs[0]]
           + [x for d in dirs[1:] for x in ("-isystem", d)] + ["-L" + d for d in libs]
           + ["-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-L" + PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, STEP)
    with open(stamp, "w") as f:
        f.write(made_for)
    return STEP


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile every source, link the shared library and the binding; return the library's path."""
    if not force and not _stale():
        build_binding()
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(max_workers=max(1, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    build_binding(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--ptxas-v" in sys.argv))
