"""Build librbq.so in-tree with nvcc for sm_100a.

Run ``python -m rotation_bit_ptq_b200.build`` (or call ``build()``).  Each
CUDA source compiles to an object under ``_build/`` (in parallel, rebuilt
when it or a header is newer than its object), then one shared library is
linked next to this file.  The CUDA runtime is linked statically.

Beside it goes _rbq_call.so, the native part of the Python binding
(csrc/rbq_call.cpp), compiled by the host compiler against the headers of the
installed torch (left out where there is none).
"""

import concurrent.futures
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "librbq.so")
# The same sources compiled with RBQ_DEBUG: device-side bounds checks on the
# indices the kernels compute (see dbg_index in csrc/rbq_sm100.cuh) record
# into the device error word instead of trapping.  Tests load it beside the
# release library; the product path never does.
LIB_DEBUG = os.path.join(PKG, "librbq_debug.so")

# The native part of the Python binding: ordinary calls without ctypes.
BINDING = os.path.join(PKG, "_rbq_call.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc():
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found")
    return path


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(obj, src, newest_header):
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return os.path.getmtime(src) > t or newest_header > t


def build(verbose=False, ptxas_info=False, jobs=None, debug=False):
    """Compile every CUDA source for sm_100a and link librbq.so (or, with
    debug=True, librbq_debug.so with -DRBQ_DEBUG, objects under _build/debug)."""
    bdir = os.path.join(BUILD, "debug") if debug else BUILD
    lib = LIB_DEBUG if debug else LIB
    os.makedirs(bdir, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    newest_header = max((os.path.getmtime(h) for h in _headers()), default=0.0)
    extra = (["-Xptxas", "-v"] if ptxas_info else []) + (["-DRBQ_DEBUG"] if debug else [])
    cmds = []
    objs = []
    for src in srcs:
        obj = os.path.join(bdir, os.path.basename(src) + ".o")
        objs.append(obj)
        if ptxas_info or _stale(obj, src, newest_header):
            cmds.append([nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with concurrent.futures.ThreadPoolExecutor(max_workers=jobs or os.cpu_count()) as ex:
        for cmd, r in ex.map(run, cmds):
            if verbose or ptxas_info or r.returncode:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode:
                raise RuntimeError(f"nvcc failed on {cmd[-3]}")
    if cmds or not os.path.exists(lib) or any(os.path.getmtime(o) > os.path.getmtime(lib) for o in objs):
        link = [nvcc(), *ARCH, "-shared", "-o", lib, *objs, "-lcudart_static", "-lrt", "-lpthread", "-ldl"]
        r = subprocess.run(link, capture_output=True, text=True)
        if verbose or r.returncode:
            sys.stderr.write(" ".join(link) + "\n" + r.stdout + r.stderr)
        if r.returncode:
            raise RuntimeError(f"link of {os.path.basename(lib)} failed")
    if not debug:
        build_binding(verbose)
    return lib


def built_for():
    """What _rbq_call.so depends on besides its source: it is compiled against the
    headers of one torch and one Python, and holds this text."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:       # a torch that was not installed as a package
        import torch
        version = torch.__version__
    return f"torch {version}, {sys.implementation.cache_tag}"


def build_binding(verbose=False):
    """Compile csrc/rbq_call.cpp to _rbq_call.so, if it is older than its source or
    was built for another torch or Python.  Without torch there is nothing to
    bind (librbq.so needs none): returns None."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        sys.stderr.write("torch is not installed: _rbq_call.so, the native part of the Python binding, is not built\n")
        return None
    src = os.path.join(CSRC, "rbq_call.cpp")
    key = built_for()
    key_file = os.path.join(BUILD, "rbq_call.key")
    if not _stale(BINDING, src, os.path.getmtime(os.path.join(INCLUDE, "rbq.h"))) and os.path.exists(key_file):
        with open(key_file) as f:
            if f.read() == key:
                return BINDING
    torch_dir = spec.submodule_search_locations[0]
    inc, libs = os.path.join(torch_dir, "include"), os.path.join(torch_dir, "lib")
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared", "-fvisibility=hidden",
           f'-DRBQ_BUILT_FOR="{key}"', "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda_inc, src, "-o", BINDING,
           "-L", libs, "-ltorch_python", "-ltorch_cpu", "-ltorch", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode:
        raise RuntimeError("g++ failed on rbq_call.cpp")
    os.makedirs(BUILD, exist_ok=True)
    with open(key_file, "w") as f:
        f.write(key)
    return BINDING


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv, debug="--debug" in sys.argv))
