"""Build ``libkvd.so`` (the C-ABI library of the decode step) for sm_103a.

Each ``csrc/*.cu`` translation unit is compiled in parallel with nvcc, then the
objects are linked into ``kv_cache_decode_append_gb300/_build/libkvd.so``
(static CUDA runtime, so the library needs only the driver at run time).
``csrc/kvd_binding.cpp`` becomes the extension module of the compiled calls,
``_build/_kvd-<torch version>.so``, linked against that library and this torch.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libkvd.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


BINDING_SRC = os.path.join(CSRC, "kvd_binding.cpp")


def binding_path() -> str:
    import torch
    return os.path.join(BUILD_DIR, f"_kvd-{torch.__version__}.so")


def _binding_compile(obj: str):
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", INCLUDE, "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-I", sysconfig.get_paths()["include"], "-I", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
            "-c", BINDING_SRC, "-o", obj]


def _binding_link(obj: str, out: str):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-shared", "-o", out, obj, "-L", BUILD_DIR, "-l:libkvd.so", "-Wl,-rpath,$ORIGIN", "-L", lib,
            f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def _binding_up_to_date() -> bool:
    path = binding_path()
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(d) <= t for d in (BINDING_SRC, os.path.join(INCLUDE, "kvd.h"), os.path.abspath(__file__)))


def _deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        [os.path.join(INCLUDE, "kvd.h"), os.path.abspath(__file__)]


def up_to_date(lib_path: str = LIB_PATH) -> bool:
    if not os.path.exists(lib_path):
        return False
    t = os.path.getmtime(lib_path)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags=(), variant: str = "") -> str:
    """Compile and link ``libkvd.so`` unless it is newer than every source.

    ``variant`` builds a separate copy with ``extra_flags`` into
    ``_build/<variant>/libkvd.so`` (the timeout test builds one with
    ``-DKVD_TIMEOUT_TEST``); the library the package loads is never replaced."""
    build_dir = os.path.join(BUILD_DIR, variant) if variant else BUILD_DIR
    lib_path = os.path.join(build_dir, "libkvd.so")
    if not force and up_to_date(lib_path):
        if not variant and not _binding_up_to_date():
            _build_binding(verbose)
        return lib_path
    os.makedirs(build_dir, exist_ok=True)
    nvcc = _nvcc()
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    bobj = os.path.join(build_dir, "kvd_binding.o")
    if not variant:
        procs.append((BINDING_SRC, subprocess.Popen(_binding_compile(bobj), stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            sys.stderr.write(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"compiling failed for {failed}")
    tmp = lib_path + ".tmp"
    subprocess.run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], check=True)
    os.replace(tmp, lib_path)
    if not variant:
        _link_binding(bobj)
    return lib_path


def _link_binding(obj: str) -> None:
    tmp = binding_path() + ".tmp"
    subprocess.run(_binding_link(obj, tmp), check=True)
    os.replace(tmp, binding_path())


def _build_binding(verbose: bool = False) -> None:
    """Compile and link the extension module alone (the library is up to date)."""
    obj = os.path.join(BUILD_DIR, "kvd_binding.o")
    cmd = _binding_compile(obj)
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    _link_binding(obj)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
