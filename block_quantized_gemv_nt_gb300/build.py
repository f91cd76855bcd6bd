"""Build libnt.so in-tree (block_quantized_gemv_nt_gb300/_build/) for sm_103a, and
nt_calls.so beside it: the torch side of some calls, against torch's headers.

Each CUDA translation unit compiles in parallel with nvcc, then one link.  libnt.so is
linked first and needs no torch; without torch it is all there is.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
SO = os.path.join(BUILD, "libnt.so")
CALLS_SRC = os.path.join(CSRC, "calls.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def _torch_version() -> str:
    """Of the torch that is installed, which is not imported for it."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        found = re.search(r"^__version__\s*=\s*['\"]([\w.+-]+)['\"]", f.read(), re.M)
    return found.group(1) if found else importlib.metadata.version("torch")


def calls_so() -> str:
    """The module for this torch and this Python, whose ABIs it holds: another's is another file."""
    return os.path.join(BUILD, f"nt_calls-torch{_torch_version()}{sysconfig.get_config_var('EXT_SUFFIX')}")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(target: str, sources: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources + [os.path.join(HERE, "..", "include", "nt.h"), os.path.abspath(__file__)])


def _stale() -> bool:
    return _older(SO, sources() + glob.glob(os.path.join(CSRC, "*.cuh")))


def _calls_stale() -> bool:
    return _older(calls_so(), [CALLS_SRC])


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None, module: bool = True) -> str:
    """What is not up to date: the library, and with `module` nt_calls.so where torch is installed."""
    lib, calls = force or _stale(), module and _torch_dir() is not None and (force or _calls_stale())
    if not lib and not calls:
        return SO
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = extra or []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stdout + r.stderr)
        return obj

    def compile_calls():
        inc = os.path.join(_torch_dir(), "include")
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
        obj = os.path.join(BUILD, "calls.o")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I" + inc, "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
               "-I" + sysconfig.get_paths()["include"], "-I" + cuda, "-c", CALLS_SRC, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on calls.cpp:\n{r.stdout}\n{r.stderr}")
        return obj

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        calls_obj = ex.submit(compile_calls) if calls else None
        objs = list(ex.map(compile_one, sources() if lib else []))
    if lib:
        tmp = SO + f".{os.getpid()}.tmp"
        run([nvcc, *ARCH, "-shared", *objs, "-o", tmp, "-lcudart"])
        os.replace(tmp, SO)
    if calls:
        tmp = calls_so() + f".{os.getpid()}.tmp"
        run(["g++", "-shared", calls_obj.result(), "-o", tmp, "-L" + os.path.join(_torch_dir(), "lib"), "-ltorch_python",
             "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L" + BUILD, "-lnt", "-Wl,-rpath,$ORIGIN"])
        os.replace(tmp, calls_so())
    return SO


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None))
