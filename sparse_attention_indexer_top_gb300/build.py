"""Build libsai.so (the C-ABI library) in-tree for sm_103a with nvcc, and the
Python module of its per-layer calls with g++.

Each ``csrc/*.cu`` translation unit is compiled in parallel to an object
file, then linked into ``libsai.so`` next to this file. Objects live in
``_build/`` (git-ignored). A unit is rebuilt when it or any header is newer
than its object. ``csrc/binding.cpp`` becomes ``_binding.so``, against the
installed torch; a stamp beside its object names the torch and the Python it
was linked for, and it is linked again when either is another.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libsai.so")
BINDING = os.path.join(HERE, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-warn-spills",
         "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _newest_header() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _binding_job(hdr: float):
    """Command that compiles binding.cpp to an object, its object, the linker's arguments, whether the object is out of
    date, and the name of the torch and the Python that it is for."""
    import torch

    abi = f"torch-{torch.__version__}-{sys.implementation.cache_tag}"
    src, obj = os.path.join(CSRC, "binding.cpp"), os.path.join(BUILD, f"binding-{abi}.o")
    top = os.path.dirname(torch.__file__)
    inc = [os.path.join(top, "include"), sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"), "/usr/local/cuda/include"]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *["-I" + i for i in inc], "-c", src, "-o", obj]
    link = ["-L" + os.path.join(top, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-L" + HERE,
            "-l:libsai.so", "-Wl,-rpath,$ORIGIN"]
    stale = not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr)
    return cmd, obj, link, stale, abi


def _read(path: str) -> str:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return ""


def build(verbose: bool = False, force: bool = False) -> str:
    """Compile and link; returns the path of libsai.so."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr = _newest_header()
    objs = []
    jobs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), hdr):
            jobs.append([nvcc, *ARCH, *FLAGS, "-c", s, "-o", o])

    cmd, bobj, link, stale, abi = _binding_job(hdr)
    if force or stale:
        jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("compiler failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        if verbose:
            sys.stderr.write(r.stdout + r.stderr)

    with cf.ThreadPoolExecutor(max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        list(ex.map(run, jobs))
    if jobs or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        tmp = LIB + ".tmp"
        run([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    stamp = os.path.join(BUILD, "binding.stamp")
    if (not os.path.exists(BINDING) or _read(stamp) != abi
            or os.path.getmtime(BINDING) < max(os.path.getmtime(bobj), os.path.getmtime(LIB))):
        tmp = BINDING + ".tmp"
        run(["g++", "-shared", "-o", tmp, bobj, *link])
        os.replace(tmp, BINDING)
        with open(stamp, "w") as f:
            f.write(abi)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
