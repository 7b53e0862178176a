"""Compile the CUDA library (csrc/*.cu, csrc/block/*.cu) for sm_103a into libbsmoe.so, in tree.

Each translation unit is compiled in parallel with nvcc; the objects are
linked into one shared library next to this file. Beside them the host compiler
builds csrc/block/calls.cpp, Python's way into include/moe_block.h, against the
installed torch. Rebuilds only what changed (object newer than its source and
every header).
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


def _calls_job(newest_header):
    """The command that builds _calls.so, or None where it is up to date (it
    belongs to one torch, whose version stands beside it)."""
    import torch
    src = os.path.join(SRC, "block", "calls.cpp")
    stamp = os.path.join(BUILD, "calls.torch")
    seen = open(stamp).read() if os.path.exists(stamp) else ""
    if seen == torch.__version__ and not _stale(CALLS, src, newest_header):
        return None
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return _calls_command(src)


def build(verbose=False, ptxas_verbose=False):
    """Build libbsmoe.so and _calls.so; returns the library's path. Raises
    RuntimeError on failure."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    sources = _sources()
    newest_header = max([os.path.getmtime(h) for h in _headers()] + [0])
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    jobs = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if ptxas_verbose or _stale(obj, src, newest_header):
            jobs.append([nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj])
    calls = _calls_job(newest_header)
    commands = jobs + ([calls] if calls else [])
    logs = []
    if commands:
        with cf.ThreadPoolExecutor(max_workers=min(12, len(commands))) as ex:
            for cmd, res in zip(commands, ex.map(lambda c: subprocess.run(c, capture_output=True, text=True),
                                                 commands)):
                logs.append(res.stdout + res.stderr)
                if res.returncode != 0:
                    if cmd is calls and os.path.exists(CALLS):
                        os.remove(CALLS)
                    raise RuntimeError("%s failed: %s\n%s" % (os.path.basename(cmd[0]), " ".join(cmd),
                                                             res.stdout + res.stderr))
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in sources]
    if jobs or not os.path.exists(LIB):
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("link failed: %s\n%s" % (" ".join(cmd), res.stdout + res.stderr))
    if verbose:
        for l in logs:
            if l.strip():
                print(l)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose=True, ptxas_verbose="-v" in sys.argv))
