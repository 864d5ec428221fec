"""Builds libsvdq.so in-tree with nvcc for sm_100a.

    python -m bit_rank_compensated_b200.build [--force] [--verbose]

Each .cu file under csrc/ is compiled to an object in _build/ (rebuilt when it or a header
changed) and linked with the static CUDA runtime into bit_rank_compensated_b200/libsvdq.so.
The eigen-solver library used by the offline prepare step is loaded at run time; the path of
the copy bundled with the installed nvidia-cusolver wheel is baked in as a hint.

csrc/binding.cpp (the Python calls of the operators around the projections) is compiled against the
installed torch into bit_rank_compensated_b200/_binding.so; without torch only the library is built.
"""
from __future__ import annotations

import argparse
import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libsvdq.so")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++20", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _cusolver_hint() -> str | None:
    try:
        import nvidia.cusolver  # type: ignore

        base = list(nvidia.cusolver.__path__)[0]
        p = os.path.join(base, "lib", "libcusolver.so.11")
        return p if os.path.exists(p) else None
    except Exception:
        return None


def _newest_header() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "svdq.h")]
    return max(os.path.getmtime(h) for h in hs)


def _binding_command(torch) -> list[str]:
    import sysconfig

    src = os.path.join(CSRC, "binding.cpp")
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    includes = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(base, "lib")
    return [shutil.which("g++") or "c++", "-O2", "-std=c++20", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-isystem{i}" for i in includes],
            f"-I{INCLUDE}", src, "-o", BINDING, f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            f"-Wl,-rpath,{lib}"]


def build_binding(force: bool = False, verbose: bool = False) -> str | None:
    """Compiles csrc/binding.cpp against the installed torch, again where it or torch or Python has changed since.
    Without torch there is nothing to bind: None."""
    try:
        import torch
    except ImportError:
        print("torch is not installed: libsvdq.so is built, the Python binding is not", file=sys.stderr)
        return None
    cmd = _binding_command(torch)
    made_for = "\n".join([torch.__version__, sys.version, *cmd])
    record = os.path.join(BUILD, "binding.txt")
    newest = max(os.path.getmtime(f) for f in (os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "svdq.h"), __file__))
    if not force and os.path.exists(BINDING) and os.path.exists(record) and os.path.getmtime(BINDING) >= newest:
        with open(record) as f:
            if f.read() == made_for:
                return BINDING
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.makedirs(BUILD, exist_ok=True)
    with open(record, "w") as f:
        f.write(made_for)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    hint = _cusolver_hint()
    defs = [f'-DSVDQ_CUSOLVER_HINT="{hint}"'] if hint else []
    hdr_t = _newest_header()
    objs, todo = [], []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if not force and os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), hdr_t):
            continue
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *defs, *(extra_flags or []), "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        todo.append(cmd)
    # the files do not depend on one another: a few compilers at a time
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(6, os.cpu_count() or 1)) as pool:
        for _ in pool.map(lambda c: subprocess.run(c, check=True), todo):
            pass
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        cmd = [nvcc, *ARCH, "-shared", "-cudart=static", "-o", LIB, *objs, "-ldl", "-lpthread"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    build_binding(force, verbose)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print register / smem usage per kernel")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_info else None
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose, extra_flags=extra))


if __name__ == "__main__":
    sys.exit(main())
