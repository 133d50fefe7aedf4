"""Build libq4k.so in-tree for GB300 (sm_103a) with nvcc.

Each ``csrc/*.cu`` file is compiled on its own (in parallel) with
``-gencode arch=compute_103a,code=sm_103a``; the objects are linked into
``q4_weight_matmul_gb300/libq4k.so`` (CUDA runtime linked statically).
``csrc/binding.cpp`` becomes the Python module ``_calls`` beside it (g++,
against the headers of the torch that imports it).
Each is made again only when a source file is newer, the module also when it
was made for another Python or torch.

    python -m q4_weight_matmul_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import concurrent.futures as cf
import fcntl
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
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libq4k.so")
PEAKS_SRC = os.path.join(CSRC, "peaks", "peaks.cu")
PEAKS_LIB = os.path.join(PKG, "libq4k_peaks.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_LIB = os.path.join(PKG, "_calls.so")
BINDING_STAMP = os.path.join(BUILD_DIR, "calls_made_for.txt")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
          "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libq4k.so")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(made, deps) -> bool:
    if not all(map(os.path.exists, made)):
        return True
    t = min(map(os.path.getmtime, made))
    return any(os.path.getmtime(p) > t for p in deps)


def _stale_lib() -> bool:
    return _older((LIB_PATH, PEAKS_LIB),
                  sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")) + [PEAKS_SRC, os.path.abspath(__file__)])


def _made_for() -> str:
    """The Python and the torch that the binding's module is compiled against."""
    import torch
    return f"python {sys.version}\ntorch {torch.__version__} in {os.path.dirname(torch.__file__)}\n"


def _stale_binding() -> bool:
    if _older((BINDING_LIB, BINDING_STAMP),
              glob.glob(os.path.join(INCLUDE, "*.h")) + [BINDING_SRC, os.path.abspath(__file__)]):
        return True
    with open(BINDING_STAMP) as f:
        return f.read() != _made_for()


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    if src == PEAKS_SRC:
        obj = os.path.join(BUILD_DIR, "peaks_probe.o")
    cmd = [nvcc(), *ARCH, *CFLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def _compile_binding() -> None:
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = f"{BINDING_LIB}.{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           *(f for d in (INCLUDE, sysconfig.get_paths()["include"], os.path.join(at, "include"),
                         os.path.join(at, "include", "torch", "csrc", "api", "include"), cuda) for f in ("-I", d)),
           BINDING_SRC, "-o", tmp, "-L", os.path.join(at, "lib"), "-Wl,-rpath," + os.path.join(at, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {os.path.basename(BINDING_SRC)} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_LIB)
    with open(BINDING_STAMP, "w") as f:
        f.write(_made_for())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source and link libq4k.so (and the benchmark's
    tensor-rate probe, libq4k_peaks.so), and the binding's module; return the
    library's path."""
    def stale():
        return force or _stale_lib(), force or _stale_binding()

    if not any(stale()):
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    # one process at a time: the others wait, and find what it made
    with open(os.path.join(BUILD_DIR, "lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        _make(*stale(), verbose)
    return LIB_PATH


def _make(lib: bool, binding: bool, verbose: bool) -> None:
    srcs = sources() + [PEAKS_SRC] if lib else []
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        made = ex.submit(_compile_binding) if binding else None
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
        if made:
            made.result()
    if not lib:
        return
    for path, members in ((LIB_PATH, objs[:-1]), (PEAKS_LIB, objs[-1:])):
        tmp = path + ".tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *members]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link of {os.path.basename(path)} failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, path)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
