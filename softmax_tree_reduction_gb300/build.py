"""Build libtreeattn.so in-tree with nvcc for sm_103a (GB300).

Each translation unit under csrc/ is compiled in parallel, then linked into
``softmax_tree_reduction_gb300/libtreeattn.so`` (static CUDA runtime, no
torch headers).  Objects go to ``softmax_tree_reduction_gb300/_build/``.

``build(debug=True)`` makes the bounds-checking library instead,
``libtreeattn_debug.so`` (objects in ``_build_debug/``): the same sources
compiled with TA_DEBUG_BOUNDS, whose kernels check computed indices against
their buffers, skip an access that falls outside and report it through the
device error word (TA_ERR_DEVICE_BOUNDS).  Point the binding at it with the
TREE_ATTN_LIBRARY environment variable.

The argument marshalling of the calls around the decode step
(csrc/serving_calls.cpp) is compiled with g++ against torch's and Python's
headers into ``softmax_tree_reduction_gb300/_serving_calls.so``, for the torch
and Python that run the build: with others it is built again.  The library
itself needs nvcc alone; without torch (``python
softmax_tree_reduction_gb300/build.py``) only it is built.

    python -m softmax_tree_reduction_gb300.build [--verbose-ptxas] [--force] [--debug]
"""
from __future__ import annotations

import os
import platform
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libtreeattn.so")
CALLS_SOURCE = os.path.join(CSRC, "serving_calls.cpp")
CALLS = os.path.join(HERE, "_serving_calls.so")
CALLS_FOR = os.path.join(BUILD, "serving_calls.for")  # what CALLS was built for
LIB_DEBUG = os.path.join(HERE, "libtreeattn_debug.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

SOURCES = ["api.cu", "combine.cu", "split_kv_mma.cu", "split_kv_fma_bf16.cu", "split_kv_fma_f32.cu",
           "noalloc.cu", "tokens.cu", "page_select.cu", "decode_selected.cu", "split_kv_fp8.cu", "split_kv_tc05.cu", "split_kv_tc05_fp8.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _torch():
    """The torch that the marshalling module is built for, or None."""
    try:
        import torch
    except ImportError:
        return None
    return torch


def _calls_for(torch) -> str:
    """Torch and Python versions, whose ABIs the module's binary depends on."""
    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')} {platform.machine()}"


def _calls_command(torch, out: str) -> list:
    """The compiler call that makes the marshalling module."""
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-I" + os.path.join(root, "include"), "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"),
            "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"), CALLS_SOURCE, "-o", out, "-L" + lib,
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ldl", "-Wl,-rpath," + lib]


def _newer(out: str, sources: list) -> bool:
    """Whether `out` exists and was made after every one of its sources."""
    return os.path.exists(out) and os.path.getmtime(out) >= max(os.path.getmtime(f) for f in sources)


def _common_sources() -> list:
    return [os.path.join(INCLUDE, "tree_attn.h"), os.path.abspath(__file__)]


def _lib_up_to_date(lib: str) -> bool:
    own = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != os.path.basename(CALLS_SOURCE)]
    return _newer(lib, own + _common_sources())


def _calls_up_to_date(torch) -> bool:
    if torch is None:  # nothing that could use it
        return True
    if not _newer(CALLS, [CALLS_SOURCE] + _common_sources()) or not os.path.exists(CALLS_FOR):
        return False
    with open(CALLS_FOR) as fh:
        return fh.read() == _calls_for(torch)


def up_to_date(lib: str = LIB) -> bool:
    return _lib_up_to_date(lib) and _calls_up_to_date(_torch())


def _start(cmd: list) -> subprocess.Popen:
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = True, debug: bool = False) -> str:
    lib = LIB_DEBUG if debug else LIB
    build_dir = BUILD + "_debug" if debug else BUILD
    torch = _torch()
    make_lib = force or not _lib_up_to_date(lib)
    make_calls = torch is not None and (force or not _calls_up_to_date(torch))
    if not make_lib and not make_calls:
        return lib
    os.makedirs(build_dir, exist_ok=True)
    os.makedirs(BUILD, exist_ok=True)
    # every command first: nothing is running yet when one cannot be made
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    if debug:
        extra.append("-DTA_DEBUG_BOUNDS")
    objs = [os.path.join(build_dir, src.replace(".cu", ".o")) for src in SOURCES]
    commands = [(src, [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj])
                for src, obj in zip(SOURCES, objs)] if make_lib else []
    calls_command = _calls_command(torch, CALLS + ".tmp") if make_calls else None
    running = [(src, cmd, _start(cmd)) for src, cmd in commands]
    calls_failed = ""
    calls = None
    if make_calls:
        try:
            calls = _start(calls_command)
        except OSError as e:
            calls_failed = str(e)
    failed = []
    for src, cmd, pr in running:
        out, _ = pr.communicate()
        if pr.returncode != 0:
            failed.append((src, out))
        elif out and (verbose_ptxas or not quiet):
            sys.stdout.write(f"--- {src}\n{out}")
    if calls is not None:
        out, _ = calls.communicate()
        if calls.returncode != 0:
            calls_failed = out
        else:
            os.replace(CALLS + ".tmp", CALLS)
            with open(CALLS_FOR, "w") as fh:
                fh.write(_calls_for(torch))
    if failed:
        msg = "\n".join(f"--- {s}\n{o}" for s, o in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    if make_lib:
        tmp = lib + ".tmp"
        subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lrt",
                        "-lpthread"], check=True)
        os.replace(tmp, lib)
    if calls_failed:  # the library is complete all the same
        raise RuntimeError(f"{calls_command[0]} failed on {os.path.basename(CALLS_SOURCE)} "
                           f"({os.path.basename(lib)} is built):\n{calls_failed}")
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--verbose-ptxas" in sys.argv, quiet=False,
                debug="--debug" in sys.argv))
