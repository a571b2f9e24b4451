"""Build libmoda.so in-tree for sm_103a (nvcc, no cmake).

    python -m sequence_depth_attention_gb300.build [--force] [--verbose]

Each .cu under csrc/ is compiled in parallel to an object, then linked into
``_build/libmoda.so`` with the CUDA runtime linked statically, so the library
depends only on the driver. Objects are rebuilt when a source or header is
newer than them. csrc/paged_py.cpp becomes the Python extension module
``_build/paged_py.so`` (g++, Python's and PyTorch's headers, no CUDA); where that
fails the library is built all the same, with a warning.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(BUILD, "libmoda.so")
EXT = os.path.join(BUILD, "paged_py.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(extra=()):
    return [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
            "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC,
            "--expt-relaxed-constexpr", *extra]


def build_extension(force: bool = False) -> str:
    """The extension module that marshals the paged calls' arguments."""
    import torch

    src = os.path.join(CSRC, "paged_py.cpp")
    stamp = EXT + ".torch"  # it is bound to the torch that it was built for
    newest = max(os.path.getmtime(p) for p in (src, os.path.join(INCLUDE, "moda.h")))
    if not force and os.path.exists(EXT) and os.path.exists(stamp) and os.path.getmtime(EXT) >= newest:
        with open(stamp) as f:
            if f.read() == torch.__version__:
                return EXT
    tmp = EXT + f".tmp{os.getpid()}"
    root = os.path.dirname(torch.__file__)
    includes = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(root, "include"),
                os.path.join(root, "include", "torch", "csrc", "api", "include")]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(x for p in includes for x in ("-isystem", p)), src, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(src)}:\n{r.stderr}")
    os.replace(tmp, EXT)
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return EXT


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
               glob.glob(os.path.join(INCLUDE, "*.h")))
    newest_header = max((os.path.getmtime(h) for h in headers), default=0)
    cc = nvcc()

    def obj_of(src):
        return os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")

    def compile_one(src):
        obj = obj_of(src)
        if (not force and os.path.exists(obj)
                and os.path.getmtime(obj) >= max(os.path.getmtime(src), newest_header)):
            return obj, ""
        cmd = [cc, *_flags(extra), "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        ext = ex.submit(build_extension, force)
        results = list(ex.map(compile_one, srcs))
        try:
            ext.result()
        except (ImportError, OSError, RuntimeError) as e:
            for stale in (EXT, EXT + ".torch"):
                if os.path.exists(stale):
                    os.remove(stale)
            warnings.warn(f"paged_py is not built, paged calls take a few us longer: {e}", RuntimeWarning)
    if verbose:
        for _, log in results:
            if log:
                print(log)
    objs = [o for o, _ in results]
    if force or not os.path.exists(LIB) or any(
            os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [cc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static",
               "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
