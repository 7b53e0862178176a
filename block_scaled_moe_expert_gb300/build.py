"""Compile the CUDA library (csrc/*.cu, csrc/block/*.cu) for sm_103a into libbsmoe.so, in tree.

Each translation unit is compiled in parallel with nvcc; the objects are
linked into one shared library next to this file; that takes the CUDA toolkit
alone. A step of its own, left out where torch is not installed, builds
csrc/block/calls.cpp (_calls.so), Python's way into include/moe_block.h, with the
host compiler against the installed torch. Rebuilds only what changed (object
newer than its source and every header).
"""
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libbsmoe.so")
CALLS = os.path.join(HERE, "_calls.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", f"-I{INCLUDE}"]


def _nvcc():
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return path


def _headers():
    return [h for d in (SRC, os.path.join(SRC, "block"), INCLUDE) for e in ("*.cuh", "*.h")
            for h in glob.glob(os.path.join(d, e))]


def _sources():
    """Every translation unit; file names are unique over the folders."""
    return sorted(glob.glob(os.path.join(SRC, "*.cu")) + glob.glob(os.path.join(SRC, "block", "*.cu")))


def _stale(obj, src, newest_header):
    return not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), newest_header)


def _calls_command(src):
    """The host compiler's line for calls.cpp."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    gxx = shutil.which("g++") or shutil.which("c++")
    if gxx is None:
        raise RuntimeError("no C++ compiler found: g++ is required to build the Python calls")
    return [gxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-DTORCH_EXTENSION_NAME=_calls",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in include], src,
            "-o", CALLS, "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def _run(cmd, what):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("%s failed: %s\n%s" % (what, " ".join(cmd), res.stdout + res.stderr))
    return res.stdout + res.stderr


def build_library(ptxas_verbose=False):
    """Build libbsmoe.so; returns the compilers' messages. Raises RuntimeError on
    failure."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    newest_header = max([os.path.getmtime(h) for h in _headers()] + [0])
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    jobs, objs = [], []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if ptxas_verbose or _stale(obj, src, newest_header):
            jobs.append([nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj])
    logs = []
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(12, len(jobs))) as ex:
            logs = list(ex.map(lambda c: _run(c, "nvcc"), jobs))
    if any(not os.path.exists(LIB) or os.path.getmtime(LIB) < os.path.getmtime(o) for o in objs):
        _run([nvcc, *ARCH, "-shared", "-o", LIB, *objs], "link")
    return logs


def build_calls():
    """Build _calls.so for the installed torch (the stamp beside it says which);
    returns its path, or None without torch. Raises RuntimeError on failure."""
    try:
        import torch
    except ImportError:
        return None
    os.makedirs(BUILD, exist_ok=True)
    src, stamp = os.path.join(SRC, "block", "calls.cpp"), os.path.join(BUILD, "calls.torch")
    seen = open(stamp).read() if os.path.exists(stamp) else ""
    newest_header = max(os.path.getmtime(h) for h in glob.glob(os.path.join(INCLUDE, "*.h")))
    if seen != torch.__version__ or _stale(CALLS, src, newest_header):
        for old in (stamp, CALLS):
            if os.path.exists(old):
                os.remove(old)
        _run(_calls_command(src), "g++")
        with open(stamp, "w") as f:
            f.write(torch.__version__)
    return CALLS


def build(verbose=False, ptxas_verbose=False):
    """Build libbsmoe.so and, with torch, _calls.so; returns the library's path.
    Raises RuntimeError on failure; the library is there all the same where only
    the calls failed."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        calls = ex.submit(build_calls)
        logs = build_library(ptxas_verbose)
        made = calls.result()
    if verbose:
        for l in logs:
            if l.strip():
                print(l)
        if made is None:
            print("torch is not installed: built without Python's calls (_calls.so)")
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose=True, ptxas_verbose="-v" in sys.argv))
