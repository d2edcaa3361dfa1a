"""Build libpwp.so (CUDA for sm_100a) in-tree with nvcc.

    python -m post_weight_pruning_b200.build          # or build() from Python

Objects go to _build/ at the repository root; the shared library is written next
to this file so the Python binding finds it.  Where PyTorch for CUDA and g++ are installed, _fastcall
(the forward operators' usual calls, marshalled without the interpreter) is built beside it;
where it cannot be, a warning says so and the binding marshals those calls itself.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(ROOT, "_build", "obj")
LIB = os.path.join(HERE, "libpwp.so")
# named for this interpreter: another one does not import it
FASTCALL = os.path.join(HERE, "_fastcall" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + os.path.join(ROOT, "include")]


def _nvcc():
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _compile(src, extra, verbose):
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    deps = [src] + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "pwp.h")]
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(d) for d in deps):
        return obj
    cmd = [_nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr.strip():
        print(r.stderr, file=sys.stderr)
    return obj


def _read(path):
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def _remove(path):
    if os.path.exists(path):
        os.remove(path)


def _build_fastcall(verbose):
    """g++ against PyTorch's headers and libpwp.so, which is found beside it at run time.  Built
    again when its sources, the command or PyTorch's version are others than those recorded
    with the objects."""
    _remove(os.path.join(HERE, "_fastcall.so"))      # a build without the interpreter's tag
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return
    torch = os.path.dirname(spec.origin)
    src = os.path.join(CSRC, "fastcall.cpp")
    header = os.path.join(ROOT, "include", "pwp.h")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    lib = os.path.join(torch, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", src, "-o", FASTCALL, *("-I" + p for p in inc), "-L" + HERE,
           "-l:libpwp.so", "-Wl,-rpath,$ORIGIN", "-L" + lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    record, built_for = os.path.join(OBJ, "fastcall.txt"), " ".join(cmd) + "\n" + (_read(os.path.join(torch, "version.py")) or "")
    if os.path.exists(FASTCALL) and _read(record) == built_for and \
            os.path.getmtime(FASTCALL) >= max(os.path.getmtime(src), os.path.getmtime(header)):
        return
    _remove(FASTCALL)          # what does not fit this PyTorch or pwp.h is not left to be loaded
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failed = f"{r.stdout}\n{r.stderr}" if r.returncode != 0 else None
    except OSError as e:
        failed = str(e)
    if failed is not None:
        _remove(FASTCALL)
        warnings.warn(f"{os.path.basename(FASTCALL)} not built, small calls of the forward operators take longer:\n{failed}")
        return
    with open(record, "w") as f:
        f.write(built_for)


def build(verbose: bool = False, extra=()) -> str:
    os.makedirs(OBJ, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, list(extra), verbose), srcs))
    newest = max(os.path.getmtime(o) for o in objs)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        cmd = [_nvcc(), *ARCH, "-shared", "-o", LIB, *objs, "-lcuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    _build_fastcall(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
