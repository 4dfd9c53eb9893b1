"""Build libdeltarule.so in-tree with nvcc for sm_100a, and the host module of calls on torch tensors."""
from __future__ import annotations

import glob
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libdeltarule.so")
CALLS = os.path.join(HERE, "_torch_calls.so")
CALLS_SRC = [os.path.join(CSRC, "torch_calls.cpp"), os.path.join(os.path.dirname(HERE), "include", "delta_rule.h")]
ROOT = os.path.dirname(HERE)

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-warn-spills",
    "-Xlinker", "-z,defs",  # an undefined symbol fails the build, not the first load
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(ROOT, "include", "*.h")))


def source_digest(files: list[str] | None = None) -> str:
    """sha256 over library sources (identifies the code a profile was taken on): every source,
    or only the named files of csrc/ (those that define one kernel and its launch)."""
    import hashlib
    h = hashlib.sha256()
    paths = sources() if files is None else [os.path.join(CSRC, f) for f in sorted(files)]
    for p in paths:
        h.update(os.path.basename(p).encode())
        with open(p, "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:16]


# the files that define each profiled kernel and its launch
KERNEL_FILES = {
    "k_bwd_chunk_tc": ["tc_bwd.cu", "tc_ptx.cuh", "tc_tile.cuh", "tc_inverse.cuh", "tc_host.cuh", "dr_common.cuh"],
}


def _key(cmd: list[str], torch) -> str:
    """What the module of calls depends on: its sources (not where they lie), the command, torch and Python."""
    import hashlib
    import sysconfig
    h = hashlib.sha256()
    for part in (*(os.path.basename(c) if c in CALLS_SRC else c for c in cmd), torch.__version__, sysconfig.get_config_var("EXT_SUFFIX") or ""):
        h.update(part.encode() + b"\0")
    for p in CALLS_SRC:
        with open(p, "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:32]


def build_calls(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/torch_calls.cpp (host code against torch's and Python's headers) into _torch_calls.so.

    The module carries the key of what it was built from; one of another torch, Python or source is built again."""
    import sysconfig

    import torch
    t = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", CALLS_SRC[0],
           "-isystem", os.path.join(t, "include"), "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, "-L" + os.path.join(t, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python",
           # torch's own C++ runtime: a second, static one would not know torch's exceptions
           "-nodefaultlibs", "-l:libstdc++.so.6", "-lm", "-lgcc_s", "-lgcc", "-lc"]
    key = _key(cmd, torch)
    if not force and os.path.exists(CALLS):
        with open(CALLS, "rb") as f:
            if key.encode() in f.read():
                return CALLS
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd += [f'-DCALLS_KEY="{key}"', "-o", tmp]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, CALLS)
    return CALLS


def build_library(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile csrc/delta_rule_lib.cu (the unity translation unit) into libdeltarule.so; needs nvcc and nothing else."""
    newest = max(os.path.getmtime(p) for p in sources())
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= newest:
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *NVCC_FLAGS, *(extra or []), "-o", tmp, os.path.join(CSRC, "delta_rule_lib.cu")]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """The library, and then the module of calls on torch tensors, where there is a torch."""
    lib = build_library(force, verbose, extra)
    try:
        import torch  # noqa: F401
    except ImportError:
        print("no torch: _torch_calls.so, the calls of the softmax-attention layers on its tensors, is not built")
        return lib
    build_calls(force, verbose)
    return lib


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, extra=["-Xptxas", "-v"] if "-v" in sys.argv else None))
