"""Build step of the CUDA library: nvcc for sm_103a, in-tree (``_build/libgdn.so``).

Each translation unit is compiled in parallel, then linked into one shared
library with the C ABI of ``include/gdn.h`` and ``include/gdn_block.h``.  Beside
them g++ compiles ``csrc/block_py.cpp``, the Python extension that checks and
allocates for the operators of ``include/gdn_block.h`` (``_build/gdn_block_py.*.so``,
one for each torch and Python that has built it).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
import warnings

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libgdn.so")
SOURCES = ["api.cu", "plan.cu", "fwd.cu", "fwd_prep_tc.cu", "fwd_tc.cu", "bwd.cu", "bwd_chain_tc.cu", "bwd_local_tc.cu",
           "recurrent.cu", "block_api.cu", "attn_rows.cu", "attn_rows_sinks.cu", "attn_rows_head.cu",
           "attn_rows_tail.cu", "attn_chunk_tc.cu", "attn_prefix.cu",
           "rope.cu", "norm_rope.cu", "pages.cu", "rmsnorm.cu", "scan.cu"]
PY_SOURCE = os.path.join(CSRC, "block_py.cpp")
# tied to the C++ ABI of one torch and one Python, so it carries both in its name
PY_LIB = os.path.join(BUILD, f"gdn_block_py.torch-{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the GB300 library needs the CUDA toolkit to build")
    return p


def _deps_mtime() -> float:
    inc = os.path.join(ROOT, "include")
    files = [os.path.join(d, f) for d in (CSRC, inc) for f in os.listdir(d)] + [__file__]
    return max(os.path.getmtime(f) for f in files)


def _fresh(path: str) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= _deps_mtime()


def _build_lib(nvcc: str, verbose: bool) -> None:
    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


def _build_py(nvcc: str) -> str:
    """Compiles the extension; returns the reason when that fails, and then leaves none of an older source behind."""
    root = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include"), os.path.join(ROOT, "include")]
    tmp = PY_LIB + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{i}" for i in inc), PY_SOURCE, "-o", tmp, f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        error = r.stderr if r.returncode != 0 else ""
    except OSError as e:
        error = str(e)
    if not error:
        os.replace(tmp, PY_LIB)
        return ""
    for f in (tmp, PY_LIB):
        if os.path.exists(f):
            os.remove(f)
    return f"g++ failed for {os.path.basename(PY_SOURCE)}:\n{error}"


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every kernel for sm_103a and link ``libgdn.so``; returns its path.

    The Python extension is compiled beside it.  Where that fails (no g++ or Python headers, another torch) there is a
    warning, and only the functions of block.py are missing: they raise at their first call."""
    os.makedirs(BUILD, exist_ok=True)
    old = [f for f in (LIB, PY_LIB) if force or not _fresh(f)]
    if not old:
        return LIB
    nvcc = _nvcc()
    with cf.ThreadPoolExecutor(1) as ex:
        py = ex.submit(_build_py, nvcc) if PY_LIB in old else None
        if LIB in old:
            _build_lib(nvcc, verbose)
        reason = py.result() if py else ""
    if reason:
        warnings.warn(f"built without the extension of the operators in block.py: {reason}", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
