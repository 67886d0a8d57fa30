"""Builds libminf.so (the sm_100a kernels and the C ABI) in-tree with nvcc, and
beside it, with g++, the torch binding of the paged calls.  The
library needs neither torch nor Python's headers: where they are missing it is
built all the same, and the build warns that the binding is not.

    python -m dynamic_sparse_attention_est_b200.build_lib [--force]
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libminf.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def cuda_include() -> str:
    """The CUDA headers of the toolkit that nvcc() belongs to."""
    found = shutil.which(nvcc())
    roots = [os.path.dirname(os.path.dirname(os.path.abspath(found)))] if found else []
    if found:
        roots.append(os.path.dirname(os.path.dirname(os.path.realpath(found))))
    roots += [os.environ.get("CUDA_HOME"), "/usr/local/cuda"]
    for root in roots:
        if root and os.path.exists(os.path.join(root, "include", "cuda_runtime_api.h")):
            return os.path.join(root, "include")
    raise RuntimeError("no CUDA headers beside nvcc, in CUDA_HOME or in /usr/local/cuda")


def cxx() -> str:
    """The system's compiler.  Not CXX: one that links a C++ runtime of its own into the module builds it
    without complaint, and the first exception it throws through torch's ends the process."""
    return "g++"


def binding_path() -> str:
    """The binding for this Python and this torch: another of either is another file."""
    import torch

    return os.path.join(PKG, f"_paged.{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}.so")


def build_binding() -> str:
    """Compiles the extension module against this interpreter's torch and links it to libminf.so."""
    import torch

    path, root = binding_path(), os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           cuda_include(), sysconfig.get_paths()["include"], INCLUDE]
    tmp = f"{path}.{os.getpid()}.tmp"
    cmd = [cxx(), "-O2", "-fPIC", "-std=c++17", "-shared", "-o", tmp,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in inc:
        cmd += ["-isystem" if d != INCLUDE else "-I", d]
    lib = os.path.join(root, "lib")
    # by name, not path: the module finds the library beside itself (which carries no soname, so
    # that programs linked by its path load it from there)
    cmd += [os.path.join(CSRC, "paged_binding.cpp"), "-L", PKG, "-l:libminf.so", "-L", lib, "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    subprocess.check_call(cmd)
    os.replace(tmp, path)
    return path


def _older(path: str, deps) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(p) > os.path.getmtime(path) for p in deps)


def _stale() -> bool:
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    return _older(LIB, deps + glob.glob(os.path.join(INCLUDE, "*.h")))


def _binding_stale() -> bool:
    return _older(binding_path(), glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compiles every .cu under csrc/ into one shared library, and the binding; returns the library's path."""
    if force or _stale():
        _build_library(verbose, ptxas_info)
    try:
        if force or _binding_stale():
            build_binding()
    except (ImportError, OSError, RuntimeError, subprocess.CalledProcessError) as e:
        warnings.warn(f"{LIB} is built; the torch binding of the paged calls is not: {e}")
    return LIB


def _build_library(verbose: bool, ptxas_info: bool) -> None:
    build_dir = os.path.join(PKG, "_build")
    os.makedirs(build_dir, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0 or (ptxas_info and out):
            sys.stderr.write(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"nvcc failed for {failed}")
    tmp = f"{LIB}.{os.getpid()}.tmp"
    link = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs]
    subprocess.check_call(link)
    os.replace(tmp, LIB)


def ensure_built() -> str:
    return build(force=False)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
