"""Build ``_build/libpagedkv.so`` from ``csrc/*.cu`` with nvcc for sm_103a, and
``_build/_pagedkv_calls.so`` from ``native/calls.cpp`` with g++.

Each translation unit compiles in its own process (in parallel), then nvcc
links the first into one shared library exporting the C ABI of
``include/pagedkv.h``; the second is the Python module that marshals the calls
of ``rope.py``, ``latent.py`` and ``q8.py`` and links that library.  Usable as
``python -m paged_kv_cache_213_gb300.build``.

The library needs nvcc alone.  Where the module does not build (no torch with CUDA,
no Python headers) a warning says so, and those calls are marshalled in Python.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libpagedkv.so")
CALLS_SRC = os.path.join(PKG, "native", "calls.cpp")
CALLS_PATH = os.path.join(OUT_DIR, "_pagedkv_calls.so")
CALLS_STAMP = os.path.join(OUT_DIR, "_pagedkv_calls.txt")  # what it was built for
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


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h"))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + _headers()


def _newer(path, deps) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(p) <= t for p in deps)


def _torch_dir():
    """The torch package's directory; None where there is none."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def calls_target():
    """The torch and the Python that the module has to be built for; None without torch."""
    where = _torch_dir()
    if where is None:
        return None
    with open(os.path.join(where, "version.py")) as f:
        version = re.search(r"^__version__ = ['\"](.*)['\"]", f.read(), flags=re.M)
    return f"torch {version.group(1) if version else '?'}, {sys.implementation.cache_tag}"


def calls_built_for():
    """What the module there is was built for; None without one."""
    try:
        with open(CALLS_STAMP) as f:
            return f.read()
    except OSError:
        return None


def _calls_up_to_date() -> bool:
    target = calls_target()
    return target is None or (calls_built_for() == target and
                              _newer(CALLS_PATH, [CALLS_SRC] + _headers()))


def up_to_date() -> bool:
    return _newer(LIB_PATH, _deps()) and _calls_up_to_date()


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


def _link_calls(obj: str, target: str) -> None:
    tmp = CALLS_PATH + f".tmp{os.getpid()}"
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, "-L", OUT_DIR, "-l:libpagedkv.so",
                        "-Wl,-rpath,$ORIGIN", "-L", os.path.join(_torch_dir(), "lib"), "-lc10",
                        "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {CALLS_PATH} failed:\n{r.stderr}")
    if os.path.exists(CALLS_STAMP):
        os.unlink(CALLS_STAMP)
    os.replace(tmp, CALLS_PATH)
    with open(tmp, "w") as f:
        f.write(target)
    os.replace(tmp, CALLS_STAMP)


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

    target = calls_target()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        calls = None
        if target is not None and (force or not _calls_up_to_date()):
            calls = ex.submit(_compile_calls)
        if force or not _newer(LIB_PATH, _deps()):
            results = list(ex.map(compile_one, _sources()))
            if verbose or ptxas_info:
                for _, log in results:
                    if log.strip():
                        print(log, file=sys.stderr)
            tmp = LIB_PATH + f".tmp{os.getpid()}"
            cmd = [cc, *ARCH, "-shared", "-o", tmp, *(o for o, _ in results)]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
            os.replace(tmp, LIB_PATH)
        if calls is not None:
            try:
                _link_calls(calls.result(), target)
            except (RuntimeError, OSError) as e:
                warnings.warn(f"{LIB_PATH} is built, the Python module beside it is not "
                              f"(rope.py, latent.py and q8.py marshal their calls in Python): {e}")
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
