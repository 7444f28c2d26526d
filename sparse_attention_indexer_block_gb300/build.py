"""Builds the indexer's CUDA library (libsaib.so) in-tree for sm_103a.

Each translation unit under ``csrc/`` is compiled by nvcc in parallel and the
objects are linked into one shared library next to this file. The CUDA runtime
is linked statically; the driver's tensor-map encoder is looked up at run time,
so the library needs no libcuda at link time. Beside it, g++ builds the module
that hands torch tensors to the library's small calls (_marshal.so), for the
Python and torch that run the build; the other calls do without it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libsaib.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
OBJECTS = os.path.join(HERE, "_build")
STAMP = os.path.join(OBJECTS, "marshal.txt")  # what _marshal.so was built for
SOURCES = ["api.cu", "prep.cu", "score_select.cu", "row_select.cu", "dcp.cu",
           "block_select.cu", "no_alloc.cu", "attend_api.cu", "attend.cu", "attend_tc.cu", "pages.cu",
           "append.cu", "tree.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the indexer library needs the CUDA toolkit to build")
    return cand


def _made_for() -> str:
    """What the marshalling module is built for: its objects' layouts are this Python's and this torch's."""
    import torch

    return f"{sysconfig.get_config_var('EXT_SUFFIX')} torch {torch.__version__} cxx11 {int(torch.compiled_with_cxx11_abi())}"


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MARSHAL) or not os.path.exists(STAMP):
        return True
    with open(STAMP) as f:
        if f.read() != _made_for():
            return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(MARSHAL))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps += [os.path.join(HERE, "..", "include", "indexer.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _marshal_command(nvcc: str, obj: str) -> list[str]:
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    return ["g++", "-std=c++17", "-O2", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
            "-isystem", sysconfig.get_path("include"), "-c", os.path.join(CSRC, "marshal.cpp"), "-o", obj]


def _link_marshal(obj: str) -> None:
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MARSHAL + f".tmp{os.getpid()}"
    subprocess.run(["g++", "-shared", "-o", tmp, obj, f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
                    "-lc10", "-ldl", "-Wl,--allow-shlib-undefined"], check=True)
    os.replace(tmp, MARSHAL)
    with open(STAMP, "w") as f:
        f.write(_made_for())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OBJECTS, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(OBJECTS, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [nvcc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    marshal = os.path.join(OBJECTS, "marshal.o")
    procs.append(("marshal.cpp", subprocess.Popen(_marshal_command(nvcc, marshal), stdout=subprocess.PIPE,
                                                  stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            sys.stderr.write(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    if [f for f in failed if f in SOURCES]:
        raise RuntimeError(f"compilation failed for {failed}")
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    if failed:
        # (the calls that pass by the module have what they need)
        raise RuntimeError(f"compilation failed for {failed}: it needs g++ and a torch with CUDA")
    _link_marshal(marshal)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
