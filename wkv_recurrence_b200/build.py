"""Build libwkv.so in-tree with nvcc for sm_100a (Blackwell B200), and _wkv_torch.so with g++.

    python -m wkv_recurrence_b200.build            # build if sources changed
    python -m wkv_recurrence_b200.build --force    # always rebuild
    python -m wkv_recurrence_b200.build --debug    # also the bounds-checked libwkv_debug.so

nvcc cross-compiles, so this runs on a machine without a GPU. The
bounds-checked variant (-DWKV_DEBUG) checks the indices of the kernels'
stores and workspace accesses and reports a violation through the status
word (WKV_ERR_BOUNDS from wkv_query_status) instead of touching memory; the
binding loads it instead of libwkv.so when WKV_LIBRARY=debug is set.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC_DIR = os.path.join(HERE, "csrc")
MAIN = os.path.join(SRC_DIR, "wkv_api.cu")
GATED = os.path.join(SRC_DIR, "wkv_gated.cu")
NORM = os.path.join(SRC_DIR, "wkv_norm.cu")
HOST = os.path.join(SRC_DIR, "wkv_host.cpp")  # host-side streaming of host-resident sequences
TORCH = os.path.join(SRC_DIR, "wkv_torch.cpp")  # the Python calling path of the newer entry points
LIB = os.path.join(HERE, "_build", "libwkv.so")
EXT = os.path.join(HERE, "_build", "_wkv_torch.so")
LIB_DEBUG = os.path.join(HERE, "_build", "libwkv_debug.so")
HEADER = os.path.join(ROOT, "include", "wkv.h")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-Xcompiler", "-Wall", "--threads", "4",
]


def _sources():
    found = [p for pat in ("*.cu", "*.cuh", "*.cpp", "*.h") for p in glob.glob(os.path.join(SRC_DIR, pat))]
    return sorted(p for p in found if p != TORCH) + [HEADER]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def build(force: bool = False, verbose: bool = False, extra_flags=(), debug: bool = False) -> str:
    out = LIB_DEBUG if debug else LIB
    newest = max(os.path.getmtime(p) for p in _sources())
    if not force and os.path.exists(out) and os.path.getmtime(out) >= newest:
        return out
    os.makedirs(os.path.dirname(out), exist_ok=True)
    tmp = out + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, *(["-DWKV_DEBUG"] if debug else []), *extra_flags, "-o", tmp, MAIN, GATED, NORM, HOST]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)
    return out


def ext_key() -> str:
    """What _wkv_torch.so is compiled against besides its sources: torch, its C++
    ABI and the interpreter. An object built for another key is not loaded."""
    import sysconfig

    import torch
    return f"torch {torch.__version__}, C++11 ABI {int(torch.compiled_with_cxx11_abi())}, {sysconfig.get_config_var('SOABI')}"


def build_ext(force: bool = False, verbose: bool = False) -> str:
    """_wkv_torch.so: host code against the installed torch's headers. Its key is
    in the object, and beside it for this check."""
    key, stamp = ext_key(), EXT + ".key"
    if (not force and os.path.exists(EXT) and os.path.getmtime(EXT) >= max(os.path.getmtime(p) for p in (TORCH, HEADER))
            and os.path.exists(stamp) and open(stamp).read() == key):
        return EXT
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.sep in nvcc() else "/usr/local/cuda"
    os.makedirs(os.path.dirname(EXT), exist_ok=True)
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f'-DWKV_EXT_KEY="{key}"',
           f"-I{base}/include", f"-I{base}/include/torch/csrc/api/include", f"-I{cuda}/include",
           f"-I{sysconfig.get_paths()['include']}", "-o", tmp, TORCH,
           f"-L{cuda}/lib64", "-lcudart", f"-L{base}/lib", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, EXT)
    with open(stamp, "w") as f:
        f.write(key)
    return EXT


def build_all(force: bool = False, verbose: bool = False):
    """Both variants and the Python calling path, compiled concurrently."""
    from concurrent.futures import ThreadPoolExecutor
    with ThreadPoolExecutor(3) as ex:
        futs = [ex.submit(build, force, verbose, (), d) for d in (False, True)]
        futs.append(ex.submit(build_ext, force, verbose))
        return [f.result() for f in futs]


if __name__ == "__main__":
    if "--debug" in sys.argv:
        print(build_all(force="--force" in sys.argv, verbose=True))
    else:
        print(build(force="--force" in sys.argv, verbose=True))
        print(build_ext(force="--force" in sys.argv, verbose=True))
