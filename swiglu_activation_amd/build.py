"""Compile the HIP library in-tree: csrc/*.hip -> libswiglu_gateup.so, the C client, and
the module that calls the library from torch tensors: csrc/torch_calls.cpp -> _torch_calls.so
(where torch, its headers and a C++ compiler are at hand; the library and the client need none
of them).

gfx950 only. Packed-fp32 instruction selection is switched off for the device
code (``-packed-fp32-ops``); the host pass prints a harmless warning about the
unknown feature.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
SRCS = [os.path.join(PKG_DIR, "csrc", "swiglu_gateup.hip"),
        os.path.join(PKG_DIR, "csrc", "swiglu_bias_scale.hip"),
        os.path.join(PKG_DIR, "csrc", "swiglu_fc1.hip"),
        os.path.join(PKG_DIR, "csrc", "swiglu_grouped.hip"),
        os.path.join(PKG_DIR, "csrc", "swiglu_ckpt8.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG_DIR, "libswiglu_gateup.so")
CALLS_SRC = os.path.join(PKG_DIR, "csrc", "torch_calls.cpp")
CALLS = os.path.join(PKG_DIR, "_torch_calls.so")     # CPython module, linked with torch
CLIENT_SRC = os.path.join(PKG_DIR, "examples", "c_abi_client.c")
CLIENT = os.path.join(PKG_DIR, "c_abi_client")       # a plain C program using the C ABI
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (needs ROCm)")


def compile_command(out: str = LIB, srcs=None, defines=()) -> list:
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-shared", "-fPIC",
           "-fvisibility=hidden", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-Wall", "-I", INCLUDE]
    cmd += [f"-D{d}" for d in defines]
    cmd += ["-o", out, *(SRCS if srcs is None else srcs)]
    return cmd


def build(verbose: bool = False) -> str:
    """Compile the library (always; a stale build is never reused). Returns its path."""
    tmp = LIB + ".tmp"
    cmd = compile_command(out=tmp)
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)
    os.replace(tmp, LIB)
    build_client(verbose)
    build_calls(verbose)
    return LIB


def build_calls(verbose: bool = False):
    """Compile the CPython module (C++17, host compiler) against the library and torch.
    Returns its path, or None, with a note on stderr, where what it needs is missing: the
    binding then makes those calls through ctypes."""
    import sysconfig

    def without(what):
        if os.path.exists(CALLS):
            os.remove(CALLS)             # of an earlier build, perhaps of another library
        print(f"_torch_calls.so is not built: {what}", file=sys.stderr)

    try:
        import torch
    except ImportError:
        return without("torch is not importable")
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        return without("no C++ compiler")
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    tdir = os.path.dirname(os.path.abspath(torch.__file__))
    for header in (os.path.join(tdir, "include", "ATen", "hip", "EmptyTensor.h"),
                   os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(header):
            return without(f"no {header}")
    tlib = os.path.join(tdir, "lib")
    tmp = CALLS + ".tmp"
    cmd = [cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-Wall",
           "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-isystem", os.path.join(tdir, "include"),
           "-isystem", os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(rocm, "include"),
           "-o", tmp, CALLS_SRC, "-L", PKG_DIR, "-lswiglu_gateup", "-L", tlib, "-ltorch_python",
           "-ltorch_cpu", "-ltorch_hip", "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + tlib]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"torch calls: build failed ({res.returncode}):\n{res.stderr}")
    if verbose and res.stderr.strip():
        print(res.stderr, file=sys.stderr)
    os.replace(tmp, CALLS)
    return CALLS


def build_client(verbose: bool = False) -> str:
    """Compile the plain C client (C11, host compiler) against the library."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        raise RuntimeError("no C compiler for the C ABI client")
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    cmd = [cc, "-O2", "-std=c11", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I", INCLUDE,
           "-I", os.path.join(rocm, "include"), "-o", CLIENT, CLIENT_SRC,
           "-L", PKG_DIR, "-lswiglu_gateup", "-L", os.path.join(rocm, "lib"), "-lamdhip64",
           "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + os.path.join(rocm, "lib")]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"C client build failed ({res.returncode}):\n{res.stderr}")
    return CLIENT


if __name__ == "__main__":
    print(build(verbose=True))
