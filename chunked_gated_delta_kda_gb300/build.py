"""Build ``libkda.so`` (the C-ABI KDA forward library) in-tree with nvcc, and
``kda_marshal.*.so``, a Python module between torch and some of its entry points.

Each ``csrc/*.cu`` is compiled for sm_103a in parallel, then linked into
``chunked_gated_delta_kda_gb300/_build/libkda.so`` against the shared CUDA
runtime; beside them ``csrc/kda_marshal.cpp`` by the host compiler against the
installed torch, whose version is part of the module's file name.  The library
needs neither torch nor its headers.  Rebuilds only when a source or header is
newer.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libkda.so")
MARSHAL_SOURCE = os.path.join(CSRC, "kda_marshal.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the KDA CUDA library cannot be built")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def marshal() -> str:
    """Path of the Python module for this torch and Python, whose C++ and C interfaces it is compiled against."""
    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(OUT, f"kda_marshal.torch-{torch.__version__}-{abi}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _newer(path, deps) -> bool:
    deps = [*deps, os.path.join(ROOT, "include", "kda.h"), os.path.abspath(__file__)]
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in deps)


def library_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")))


def marshal_up_to_date() -> bool:
    return _newer(marshal(), [MARSHAL_SOURCE])


def up_to_date() -> bool:
    return library_up_to_date() and marshal_up_to_date()


def _marshal_commands():
    """Compiling the Python module, and linking it beside ``libkda.so``."""
    import torch
    at = os.path.dirname(torch.__file__)
    include = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include"),
               os.path.join(ROOT, "include")]
    obj = os.path.join(OUT, "kda_marshal.o")
    host = os.environ.get("CXX") or shutil.which("g++") or "c++"
    compile_ = [host, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                *(f"-I{p}" for p in include), "-c", MARSHAL_SOURCE, "-o", obj]
    libs = os.path.join(at, "lib")
    link = [host, "-shared", "-o", marshal() + f".tmp{os.getpid()}", obj, f"-L{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-ltorch_cuda", "-lc10", "-lc10_cuda", LIB, "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    return compile_, link


def _start(cmd, verbose):
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish(procs, show) -> None:
    """Wait for the compilers [(source, process)]; raises what failed."""
    failed = []
    for src, pr in procs:
        text = pr.communicate()[0].decode(errors="replace")
        if pr.returncode != 0:
            failed.append(f"--- {src}\n{text}")
        elif show:
            print(text, file=sys.stderr)
    if failed:
        raise RuntimeError("compiling failed:\n" + "\n".join(failed))


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """``libkda.so``, which needs nvcc alone."""
    if not force and library_up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OUT, exist_ok=True)
    procs, objs = [], []
    for src in sources():
        objs.append(os.path.join(OUT, os.path.basename(src)[:-3] + ".o"))
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", objs[-1]]
        if ptxas_info:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, _start(cmd, verbose)))
    _finish(procs, verbose or ptxas_info)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, "-Xlinker", "-soname=libkda.so", *objs], check=True)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """The library and the Python module, compiled beside each other.  A module that does not compile raises when the
    library is there."""
    beside = None
    if force or not marshal_up_to_date():
        os.makedirs(OUT, exist_ok=True)
        compile_, link = _marshal_commands()
        beside = _start(compile_, verbose)
    try:
        build_library(force, verbose, ptxas_info)
    finally:
        if beside:
            _finish([("kda_marshal.cpp", beside)], verbose)
    if beside:
        subprocess.run(link, check=True)
        os.replace(link[3], marshal())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
