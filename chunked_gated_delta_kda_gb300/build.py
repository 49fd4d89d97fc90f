"""Build ``libkda.so`` (the C-ABI KDA forward library) in-tree with nvcc, and
``kda_marshal.so``, a Python module between torch and some of its entry points.

Each ``csrc/*.cu`` is compiled for sm_103a in parallel, then linked into
``chunked_gated_delta_kda_gb300/_build/libkda.so`` against the shared CUDA
runtime; beside them ``csrc/kda_marshal.cpp`` by the host compiler against the
installed torch.  Rebuilds only when a source or header is newer.
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
MARSHAL = os.path.join(OUT, "kda_marshal.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the KDA CUDA library cannot be built")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "kda.h"),
                                                                  os.path.join(CSRC, "kda_marshal.cpp"), os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(MARSHAL)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(MARSHAL))
    return all(os.path.getmtime(f) <= t for f in _deps())


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
                *(f"-I{p}" for p in include), "-c", os.path.join(CSRC, "kda_marshal.cpp"), "-o", obj]
    libs = os.path.join(at, "lib")
    link = [host, "-shared", "-o", MARSHAL + f".tmp{os.getpid()}", obj, f"-L{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-ltorch_cuda", "-lc10", "-lc10_cuda", LIB, "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    return compile_, link


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OUT, exist_ok=True)
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(OUT, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        if ptxas_info:
            cmd.insert(1, "-Xptxas=-v")
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    compile_, link = _marshal_commands()
    procs.append(("kda_marshal.cpp", subprocess.Popen(compile_, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, pr in procs:
        out, _ = pr.communicate()
        text = out.decode(errors="replace")
        if pr.returncode != 0:
            failed.append((src, text))
        elif verbose or ptxas_info:
            print(text, file=sys.stderr)
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError(f"compiling failed:\n{msg}")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, "-Xlinker", "-soname=libkda.so", *objs]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    subprocess.run(link, check=True)
    os.replace(link[3], MARSHAL)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
