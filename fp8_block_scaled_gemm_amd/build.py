"""Build the gfx950 HIP library libdgfp8.so in-tree with hipcc, and the
compiled Python binding of its operators, _binding.so, with the host compiler.

Usage: python -m fp8_block_scaled_gemm_amd.build   (or call build());
with --library only the library, which needs neither torch nor a host compiler.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import time

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libdgfp8.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["api.hip", "gemm.hip", "quantize.hip", "api_ops.hip", "router.hip", "moe.hip", "lora.hip",
           "api_experts.hip", "experts.hip", "int8.hip"]
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build the HIP library)")


def compile_flags() -> list[str]:
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
        # no packed fp32 instructions in any kernel
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wall", "-Wno-unused-command-line-argument",
        f"-I{INCLUDE}", f"-I{CSRC}",
    ]


def build(verbose: bool = False, jobs: int = 6) -> str:
    """Compile and link the library and the binding, always anew; neither is
    replaced before both are built."""
    lib = _link_library(verbose, jobs)
    binding = _link_binding(lib, verbose)
    os.replace(lib, LIB)
    os.replace(binding, BINDING)
    return LIB


def build_library(verbose: bool = False, jobs: int = 6) -> str:
    """The library alone, for callers of the C ABI."""
    os.replace(_link_library(verbose, jobs), LIB)
    return LIB


def build_binding(verbose: bool = False) -> str:
    """The binding alone, for the library that is there."""
    os.replace(_link_binding(LIB, verbose), BINDING)
    return BINDING


def _link_library(verbose: bool, jobs: int) -> str:
    """Compile every source to an object in parallel and link them; the path
    of the result, which is not in its place yet."""
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    cc = hipcc()
    # Each compiler writes its messages to a log file, not a pipe: a pipe
    # nobody drains blocks a compiler with many warnings while another one is
    # being waited for.
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".hip", ".o"))
        objs.append(obj)
        cmd = [cc, *compile_flags(), "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        log = open(obj + ".log", "w+")
        procs.append((src, subprocess.Popen(cmd, stdout=log, stderr=subprocess.STDOUT), log))
        while len([p for p in procs if p[1].poll() is None]) >= jobs:
            time.sleep(0.05)
    failed = []
    for src, p, log in procs:
        p.wait()
        log.seek(0)
        text = log.read()
        log.close()
        # hipcc's host pass does not know the packed-fp32 target feature
        lines = [l for l in text.splitlines() if "packed-fp32-ops" not in l and l.strip()]
        if p.returncode != 0:
            failed.append(src)
            print(text, file=sys.stderr)
        elif verbose and lines:
            print("\n".join(lines))
    if failed:
        raise RuntimeError(f"hipcc failed for {failed}")
    tmp = LIB + ".tmp"
    cmd = [cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", f"-Wl,-soname,{os.path.basename(LIB)}", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    return tmp


def _link_binding(lib: str, verbose: bool) -> str:
    """Compile csrc/binding.cpp against torch and link it to the library,
    which it finds beside itself; the path of the result."""
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths

    rocm = os.path.dirname(os.path.dirname(hipcc()))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{p}" for p in include_paths()), f"-I{os.path.join(rocm, 'include')}",
           f"-I{sysconfig.get_paths()['include']}", f"-I{INCLUDE}", f"-I{CSRC}", os.path.join(CSRC, "binding.cpp"),
           "-o", BINDING + ".tmp", *(f"-L{p}" for p in library_paths()), "-lc10", "-ltorch_cpu", "-ltorch_python",
           lib, f"-L{os.path.join(rocm, 'lib')}", "-lamdhip64", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    return BINDING + ".tmp"


if __name__ == "__main__":
    print(build_library(verbose=True) if "--library" in sys.argv[1:] else build(verbose=True))
