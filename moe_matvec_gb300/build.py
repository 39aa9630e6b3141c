"""Builds libqmv.so (the C-ABI library) in-tree with nvcc for sm_103a.

Every .cu unit under csrc/ is compiled in parallel, then linked into
moe_matvec_gb300/_build/libqmv.so.  Rebuilds only when a source is newer than
the library.  build(debug=True) compiles the same sources with QMV_DEBUG (the
kernels' software range checks, see qmv_debug_shrink_outputs in qmv.h) into
moe_matvec_gb300/_build_debug/libqmv_debug.so.  build_binding(name) compiles a
CPython binding (csrc/binding.cpp, csrc/binding_step.cpp) against the installed
PyTorch with g++ into moe_matvec_gb300/_build/<name>.so."""
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
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libqmv.so")
BUILD_DEBUG = os.path.join(HERE, "_build_debug")
LIB_DEBUG = os.path.join(BUILD_DEBUG, "libqmv_debug.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
          "-I", os.path.join(ROOT, "include")]
# Units whose fp64 arithmetic must not be contracted into FMAs.
NO_FMAD = {"quantize_weights.cu"}


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + [
        os.path.join(ROOT, "include", "qmv.h")]


def up_to_date(debug: bool = False) -> bool:
    lib = LIB_DEBUG if debug else LIB
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False, debug: bool = False) -> str:
    lib, bdir = (LIB_DEBUG, BUILD_DEBUG) if debug else (LIB, BUILD)
    if not force and up_to_date(debug):
        return lib
    os.makedirs(bdir, exist_ok=True)
    nvcc = _nvcc()
    flags = COMMON + (["-DQMV_DEBUG"] if debug else [])

    def compile_one(src):
        obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj]
        if os.path.basename(src) in NO_FMAD:
            cmd.insert(1, "-fmad=false")
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj, r.stderr

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        results = list(ex.map(compile_one, srcs))
    if verbose:
        for _, err in results:
            if err:
                sys.stderr.write(err)
    tmp = lib + f".{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp] + [o for o, _ in results] + ["-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


BINDINGS = {"_binding": "binding.cpp", "_binding_step": "binding_step.cpp"}


def build_binding(name: str = "_binding", force: bool = False) -> str:
    import torch
    from torch.utils import cpp_extension
    src, lib = os.path.join(CSRC, BINDINGS[name]), os.path.join(BUILD, name + ".so")
    deps = [src, os.path.join(CSRC, "binding_util.h"), os.path.join(ROOT, "include", "qmv.h"), torch.__file__]
    if not force and os.path.exists(lib) and all(os.path.getmtime(d) <= os.path.getmtime(lib) for d in deps):
        return lib
    os.makedirs(BUILD, exist_ok=True)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [os.path.join(ROOT, "include"), *cpp_extension.include_paths(), os.path.join(cuda, "include"),
           sysconfig.get_paths()["include"]]
    tmp = lib + f".{os.getpid()}.tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall", "-Wno-unused-function",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", src, "-o", tmp]
    for d in inc:
        cmd += ["-isystem" if "torch" in d else "-I", d]
    cmd += ["-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def build_bindings() -> None:
    with cf.ThreadPoolExecutor(max_workers=len(BINDINGS)) as ex:
        list(ex.map(build_binding, BINDINGS))


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="-v" in sys.argv, debug="--debug" in sys.argv))
