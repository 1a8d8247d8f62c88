"""Build libmoe_gb300.so for sm_103a with nvcc (in-tree, no torch extension).

Each .cu is compiled to an object in parallel, then linked into a shared
library next to this file; beside it the extension module ``_binding`` (the
tensor-level calls) is compiled with g++ against the installed torch.  Each is
rebuilt only when a source or header is newer, the extension also when it was
built for another torch or Python.  The library needs neither: where the
extension's headers or its compiler are missing, it is left out with a note, and
the tensor-level calls say so when they are made.
"""
from __future__ import annotations

import concurrent.futures
import glob
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
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_gb300.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_STAMP = os.path.join(BUILD, "binding.txt")  # what it was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-Werror=implicit-fallthrough", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    raise RuntimeError("nvcc not found")


def cuda_home() -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(nvcc()) or nvcc())))


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) +
            [os.path.abspath(__file__)])


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    with concurrent.futures.ThreadPoolExecutor(1) as ex:
        binding = ex.submit(build_binding, force)
        if force or stale():
            _build(BUILD, LIB, [], verbose, ptxas_info)
        binding.result()
    return LIB


def _torch_home():
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def binding_lacks():
    """What the extension cannot be built without and this machine lacks, or None."""
    home = _torch_home()
    if home is None:
        return "torch"
    for path in (os.path.join(sysconfig.get_paths()["include"], "Python.h"),
                 os.path.join(home, "include", "c10", "cuda", "CUDAGuard.h"),
                 os.path.join(cuda_home(), "include", "cuda_runtime_api.h")):
        if not os.path.exists(path):
            return path
    cxx = os.environ.get("CXX", "g++")
    return None if shutil.which(cxx) else cxx


def binding_target() -> str:
    """The torch and the Python that the extension is built for."""
    home = _torch_home()
    with open(os.path.join(home, "version.py")) as f:
        return "%s\n%s\n%s" % (sysconfig.get_config_var("SOABI"), home, f.read())


def build_binding(force: bool = False):
    """The extension module of the tensor-level calls, against this torch; None
    where something that it needs is missing."""
    lacks = binding_lacks()
    if lacks:
        sys.stderr.write("sparse_moe_decode_gb300: no %s, so the tensor-level calls of the gated "
                         "delta rule and the norms are not built\n" % lacks)
        return None
    deps = [BINDING_SRC, os.path.join(INCLUDE, "moe_gb300.h"), os.path.abspath(__file__)]
    target = binding_target()
    built_for = None
    if os.path.exists(BINDING_STAMP):
        with open(BINDING_STAMP) as f:
            built_for = f.read()
    if (not force and os.path.exists(BINDING) and built_for == target and
            all(os.path.getmtime(p) <= os.path.getmtime(BINDING) for p in deps)):
        return BINDING
    import torch
    home = _torch_home()
    tmp = BINDING + ".%d.tmp" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           "-I", INCLUDE, "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda_home(), "include"),
           BINDING_SRC, "-o", tmp, "-L", os.path.join(home, "lib"),
           "-Wl,-rpath," + os.path.join(home, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on %s:\n%s%s" % (BINDING_SRC, r.stdout, r.stderr))
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(BINDING_STAMP), exist_ok=True)
    with open(BINDING_STAMP, "w") as f:
        f.write(target)
    return BINDING


def build_variant(name: str, defines: dict) -> str:
    """A test-only copy of the library compiled with extra -D definitions
    (e.g. MOE_SABOTAGE), under _build/<name>/; never the product library."""
    out = os.path.join(BUILD, name)
    lib = os.path.join(out, "libmoe_gb300_%s.so" % name)
    if os.path.exists(lib) and all(os.path.getmtime(p) <= os.path.getmtime(lib) for p in _deps()):
        return lib
    return _build(out, lib, ["-D%s=%s" % (k, v) for k, v in sorted(defines.items())])


def _build(build_dir: str, lib_path: str, defs, verbose: bool = False,
           ptxas_info: bool = False) -> str:
    os.makedirs(build_dir, exist_ok=True)
    cc = nvcc()
    extra = (["-Xptxas", "-v"] if ptxas_info else []) + list(defs)

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        return obj, r.stdout + r.stderr

    with concurrent.futures.ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, sources()))
    if verbose or ptxas_info:
        for _, log in results:
            if log.strip():
                sys.stderr.write(log)
    tmp = lib_path + ".%d.tmp" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
