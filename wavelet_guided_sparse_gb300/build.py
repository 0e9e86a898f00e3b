"""Builds the CUDA library ``libwavefilter.so`` in-tree for sm_103a.

Each ``csrc/*.cu`` translation unit is compiled by nvcc in parallel, then the
objects are linked into one shared library next to this file.  Only the
``compute_103a``/``sm_103a`` target is generated.  ``csrc/wf_torch.cpp``, the
compiled argument marshalling of the small calls, becomes the Python module
``_wf_torch`` beside it (host code only, against the installed torch).  The
library needs no torch: where none is installed it is all that is built.
"""

from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libwavefilter.so")
MODULE = os.path.join(PKG, "_wf_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
         "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _module_flags(nvcc: str):
    """Include and link flags of the Python module; None without torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch = os.path.dirname(spec.origin)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    inc = [os.path.join(ROOT, "include"), os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"), cuda,
           sysconfig.get_paths()["include"]]
    return ([f for d in inc for f in ("-I", d)],
            ["-L", PKG, "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
             "-lc10_cuda", "-l:libwavefilter.so", "-Wl,-rpath,$ORIGIN"])


def _run(what: str, cmd, verbose: bool) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stderr}")
    if verbose and res.stderr:
        sys.stderr.write(res.stderr)


def build(verbose: bool = False, extra_flags=()) -> str:
    """Compile every kernel source and link ``libwavefilter.so``, then (where torch is
    installed) ``_wf_torch.so``; returns the library's path."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()

    module = _module_flags(nvcc)
    marshal = os.path.join(BUILD, "wf_torch.o")

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        _run(f"nvcc on {os.path.basename(src)}",
             [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj], verbose)
        return obj

    def compile_module():
        _run("g++ on wf_torch.cpp", ["g++", "-O2", "-std=c++17", "-fPIC", *module[0], "-c",
                                     os.path.join(CSRC, "wf_torch.cpp"), "-o", marshal], verbose)

    # The longest units first.
    srcs.sort(key=os.path.getsize, reverse=True)
    srcs.sort(key=lambda f: "paged" not in os.path.basename(f))
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(16, len(srcs) + 1)) as pool:
        host = pool.submit(compile_module) if module is not None else None
        objs = list(pool.map(compile_one, srcs))
    tmp = LIB + ".tmp"
    _run("link", [nvcc, *ARCH, "-shared", "-o", tmp, *objs], verbose)
    os.replace(tmp, LIB)
    if host is not None:
        host.result()
        tmp = MODULE + ".tmp"
        _run("link of the module", ["g++", "-shared", "-o", tmp, marshal, *module[1]], verbose)
        os.replace(tmp, MODULE)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
