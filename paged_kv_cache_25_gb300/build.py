"""Builds libpa.so in-tree for sm_103a with nvcc (no cmake, no torch).

Each translation unit compiles in parallel; the shared library links the CUDA
runtime statically and reaches the driver's tensor-map encoder through the
runtime's entry-point query, so it needs no -lcuda at link time.

Where torch is installed, _pa_marshal.so is built beside it: the argument
marshalling of the serving calls for Python, C++ against torch's headers.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libpa.so")
MARSHAL = os.path.join(OUT, "_pa_marshal.so")
MARSHAL_SOURCE = "marshal.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CUDA_SOURCES = ["api.cu", "cache_write.cu", "cache_rope.cu", "copy_blocks.cu", "decode.cu", "decode_verify.cu", "decode_scored.cu", "decode_scored_simt.cu", "decode_wide.cu",
                "decode_no_alloc.cu", "prefill_tc.cu", "prefill_scored.cu", "prefix_pass.cu", "prefill_scored_bias.cu", "prefill_split.cu", "prefill_split_bias.cu", "prefill_wide.cu"]
CXX_SOURCES = ["host_alloc.cpp", "prefix_cache.cpp", "rope_table.cpp", "prefix_groups.cpp"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _stale(target: str, sources) -> bool:
    """Whether target is older than its sources, the C header or this file."""
    files = [os.path.join(SRC, f) for f in sources]
    files += [os.path.join(os.path.dirname(HERE), "include", "pa.h"), os.path.abspath(__file__)]
    return not os.path.exists(target) or any(os.path.getmtime(f) > os.path.getmtime(target) for f in files)


def _has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def _torch_flags(nvcc: str):
    """(compile, link) flags for a Python extension against the installed torch."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return ([x for i in inc for x in ("-isystem", i)] + [f"-D_GLIBCXX_USE_CXX11_ABI={abi}"],
            ["-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"])


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    lib = force or _stale(LIB, [f for f in os.listdir(SRC) if f != MARSHAL_SOURCE])
    marshal = _has_torch() and (force or _stale(MARSHAL, [MARSHAL_SOURCE]))
    if not (lib or marshal):
        return LIB
    os.makedirs(OUT, exist_ok=True)
    nvcc = _nvcc()
    common = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(os.path.dirname(HERE), "include")]
    source = lambda f: os.path.join(SRC, f)            # noqa: E731
    obj = lambda f: os.path.join(OUT, f + ".o")        # noqa: E731
    cmds = {}
    if lib:
        for f in CUDA_SOURCES:
            cmds[f] = [nvcc, *ARCH, "-lineinfo", *common, "-c", source(f), "-o", obj(f)]
            if ptxas_info:
                cmds[f] += ["-Xptxas", "-v"]
        for f in CXX_SOURCES:
            cmds[f] = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", source(f), "-o", obj(f)]
    if marshal:
        cflags, ldflags = _torch_flags(nvcc)
        cmds[MARSHAL_SOURCE] = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *cflags, "-c",
                                source(MARSHAL_SOURCE), "-o", obj(MARSHAL_SOURCE)]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        return subprocess.run(cmd, capture_output=True, text=True)

    with ThreadPoolExecutor(max(1, min(len(cmds), os.cpu_count() or 1))) as ex:
        results = dict(zip(cmds, ex.map(run, cmds.values())))

    def link(target, cmd, sources):
        for f in sources:
            p = results[f]
            if p.returncode != 0:
                sys.stderr.write(p.stdout + p.stderr)
                raise RuntimeError(f"compile failed: {' '.join(cmds[f])}")
            if (verbose or ptxas_info) and (p.stdout or p.stderr):
                sys.stderr.write(p.stdout + p.stderr)
        tmp = target + f".{os.getpid()}.tmp"
        cmd = [*cmd, "-o", tmp]
        p = subprocess.run(cmd, capture_output=True, text=True)
        if p.returncode != 0:
            sys.stderr.write(p.stdout + p.stderr)
            raise RuntimeError("link failed: " + " ".join(cmd))
        os.replace(tmp, target)

    if lib:
        sources = CUDA_SOURCES + CXX_SOURCES
        link(LIB, [nvcc, *ARCH, "-shared", *map(obj, sources)], sources)
    if marshal:    # (takes the library's functions by address; torch's libraries are loaded before it)
        link(MARSHAL, ["g++", "-shared", obj(MARSHAL_SOURCE), *ldflags], [MARSHAL_SOURCE])
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
