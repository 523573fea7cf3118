"""Build the CUDA library in-tree: csrc/*.cu -> activation_sparse_gated_gb300/libsffn.so.

nvcc compiles each translation unit for sm_103a (one -gencode, -lineinfo) in
parallel, then links a shared library with the CUDA runtime linked statically.
``build_torch_calls`` compiles binding/torch_calls.cpp (host code, against the
installed PyTorch's headers) -> _torch_calls.*.so, the tensor operators' calls.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsffn.so")
# debug build: every gathered unit index and list length checked on the device
# (-DSFFN_DEBUG); a violation is reported as SFFN_ERR_DEVICE
DEBUG_LIB = os.path.join(PKG, "libsffn_debug.so")

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags=(), debug: bool = False) -> str:
    """Compile libsffn.so (or, with debug=True, libsffn_debug.so with -DSFFN_DEBUG)."""
    lib = DEBUG_LIB if debug else LIB
    if debug:
        extra_flags = tuple(extra_flags) + ("-DSFFN_DEBUG",)
    if not force and up_to_date(lib):
        return lib
    bdir = os.path.join(BUILD, "debug") if debug else BUILD
    os.makedirs(bdir, exist_ok=True)
    objs = []
    cmds = []
    for src in _sources():
        obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmds.append([NVCC, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode:
            raise RuntimeError(f"nvcc failed on {cmd[-3]}")
        return r

    with ThreadPoolExecutor(max_workers=min(8, len(cmds))) as ex:
        list(ex.map(run, cmds))
    tmp = lib + f".tmp{os.getpid()}"
    run([NVCC, *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, lib)
    return lib


# the tensor operators' calls, a CPython module against the installed PyTorch
TORCH_CALLS_SRC = os.path.join(PKG, "binding", "torch_calls.cpp")


def _torch_dir():
    """The installed PyTorch's directory; None without one that has CUDA.  (It is not imported.)"""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    d = os.path.dirname(spec.origin)
    return d if os.path.exists(os.path.join(d, "lib", "libtorch_cuda.so")) else None


def torch_calls_path() -> str:
    """Where the module for this Python and the installed PyTorch is.  It reads tensors by the layout in that PyTorch's
    headers, so its name holds both versions and another's is never loaded."""
    version, d = "none", _torch_dir()
    if d is not None:
        try:
            with open(os.path.join(d, "version.py")) as f:
                version = re.search(r"^__version__ = ['\"]([^'\"/]+)", f.read(), re.M).group(1)
        except (OSError, AttributeError):  # an unusual install: its directory's name in place of a version
            version = re.sub(r"\W", "_", d)
    return os.path.join(PKG, f"_torch_calls.torch{version}.{sysconfig.get_config_var('SOABI')}.so")


TORCH_CALLS = torch_calls_path()


def build_torch_calls(force: bool = False):
    """Compile TORCH_CALLS next to the package (a few seconds).  Without a PyTorch that has CUDA there is nothing to
    build it against: None, and the tensor operators go without it."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        sys.stderr.write("no PyTorch with CUDA: torch_calls.cpp is not built\n")
        return None
    deps = [TORCH_CALLS_SRC, os.path.abspath(__file__), *glob.glob(os.path.join(INCLUDE, "*.h"))]
    if not force and os.path.exists(TORCH_CALLS) and \
            all(os.path.getmtime(p) <= os.path.getmtime(TORCH_CALLS) for p in deps):
        return TORCH_CALLS
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = TORCH_CALLS + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I", INCLUDE,
           "-isystem", os.path.join(torch_dir, "include"),
           "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           TORCH_CALLS_SRC, "-o", tmp, "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("the host compiler failed on torch_calls.cpp")
    os.replace(tmp, TORCH_CALLS)
    return TORCH_CALLS


def main(argv) -> None:
    print(build(force="--force" in argv, verbose="-v" in argv, debug="--debug" in argv))  # needs no PyTorch
    print(build_torch_calls(force="--force" in argv))


if __name__ == "__main__":
    main(sys.argv)
