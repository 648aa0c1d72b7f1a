"""Build ``_build/libpagedkv.so`` from ``csrc/*.cu`` with nvcc for sm_103a, and
``_build/_pagedkv_calls.so`` from ``native/calls.cpp`` with g++.

Each translation unit compiles in its own process (in parallel), then nvcc
links the first into one shared library exporting the C ABI of
``include/pagedkv.h``; the second is the Python module that marshals the calls
of ``rope.py`` and ``latent.py`` and links that library.  Usable as
``python -m paged_kv_cache_213_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libpagedkv.so")
CALLS_SRC = os.path.join(PKG, "native", "calls.cpp")
CALLS_PATH = os.path.join(OUT_DIR, "_pagedkv_calls.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]
# extra nvcc flags (e.g. -D tuning macros) from the environment
NVCC_FLAGS += os.environ.get("PKV_NVCC_FLAGS", "").split()


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedkv")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [CALLS_SRC]


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(CALLS_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(CALLS_PATH))
    return all(os.path.getmtime(p) <= t for p in _deps())


def _torch_dir() -> str:
    import importlib.util
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _compile_calls() -> str:
    obj, torch_dir = os.path.join(OUT_DIR, "calls.o"), _torch_dir()
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-fPIC", "-c", CALLS_SRC, "-o", obj, "-I", INCLUDE,
                        "-I", os.path.join(torch_dir, "include"),
                        "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                        "-I", sysconfig.get_paths()["include"], "-I", cuda],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {CALLS_SRC}:\n{r.stderr}")
    return obj


def _link_calls(obj: str) -> None:
    tmp = CALLS_PATH + f".tmp{os.getpid()}"
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, "-L", OUT_DIR, "-l:libpagedkv.so",
                        "-Wl,-rpath,$ORIGIN", "-L", os.path.join(_torch_dir(), "lib"), "-lc10",
                        "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {CALLS_PATH} failed:\n{r.stderr}")
    os.replace(tmp, CALLS_PATH)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        calls = ex.submit(_compile_calls)
        results = list(ex.map(compile_one, _sources()))
        calls_obj = calls.result()
    objs = [o for o, _ in results]
    if verbose or ptxas_info:
        for _, log in results:
            if log.strip():
                print(log, file=sys.stderr)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    _link_calls(calls_obj)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
