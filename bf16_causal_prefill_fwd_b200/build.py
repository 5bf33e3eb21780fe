"""Build libb200attn.so in-tree with nvcc for sm_100a, and _paged_binding.so.

    python -m bf16_causal_prefill_fwd_b200.build [--force] [--verbose] [--trace]

The library is two translation units (csrc/b200attn.cu and csrc/paged.cu),
compiled side by side, with the CUDA runtime linked statically, so it loads
next to any PyTorch build. _paged_binding.so (csrc/paged_binding.cpp) is the
compiled part of the paged-cache operators' Python binding, built against the
installed PyTorch; it calls the library and holds no kernels.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libb200attn.so")
TRACE_LIB_PATH = os.path.join(LIB_DIR, "libb200attn_trace.so")  # same library with -DATTN_TRACE
BINDING_PATH = os.path.join(LIB_DIR, "_paged_binding.so")
HEADER = os.path.join(ROOT, "include", "b200attn.h")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-cudart", "static",
    "--expt-relaxed-constexpr",
]
UNITS = ["b200attn.cu", "paged.cu"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.h")) + [HEADER])


def up_to_date(path: str = LIB_PATH) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(s) <= t for s in sources())


def _binding_cmd(out: str) -> list[str]:
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    return [shutil.which("g++") or "g++", "-O2", "-std=c++20", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + os.path.join(root, "include"),
            "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"), "-I" + cuda,
            "-I" + sysconfig.get_paths()["include"], os.path.join(CSRC, "paged_binding.cpp"), "-o", out,
            "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]


def binding_built_for() -> str:
    """What _paged_binding.so is compiled against besides its sources: it uses PyTorch's C++ classes and
    Python's headers, whose layouts change with their versions. Kept beside it, in _paged_binding.so.stamp."""
    import torch

    return f"torch {torch.__version__} cxx11abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} python {sys.version.split()[0]}"


def binding_stamp() -> str | None:
    """What the _paged_binding.so that is there was built for; None if nothing says."""
    try:
        with open(BINDING_PATH + ".stamp") as f:
            return f.read().strip()
    except OSError:
        return None


def build_binding(force: bool = False) -> str:
    """Build lib/_paged_binding.so, if it is older than its sources or built for another PyTorch or Python."""
    src = [os.path.join(CSRC, "paged_binding.cpp"), HEADER]
    if not force and os.path.exists(BINDING_PATH) and binding_stamp() == binding_built_for() and all(
            os.path.getmtime(s) <= os.path.getmtime(BINDING_PATH) for s in src):
        return BINDING_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    res = subprocess.run(_binding_cmd(tmp), capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("g++ failed building _paged_binding.so")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_PATH + ".stamp", "w") as f:
        f.write(binding_built_for() + "\n")
    return BINDING_PATH


def build(force: bool = False, verbose: bool = False, trace: bool = False) -> str:
    """Build lib/libb200attn.so, or with trace=True lib/libb200attn_trace.so (the
    kernels record per-block events for b200attn_trace_read)."""
    path = TRACE_LIB_PATH if trace else LIB_PATH
    build_binding(force)
    if not force and up_to_date(path):
        return path
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = path + f".tmp{os.getpid()}"
    objs, procs = [], []
    try:
        for unit in UNITS:
            objs.append(f"{tmp}.{unit}.o")
            cmd = [_nvcc(), *NVCC_FLAGS, "-c", "-o", objs[-1], os.path.join(CSRC, unit)]
            if trace:
                cmd += ["-DATTN_TRACE"]
            if verbose:
                cmd += ["-Xptxas", "-v"]
            procs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
        logs = [p.communicate()[0] for p in procs]
        if all(p.returncode == 0 for p in procs):
            link = subprocess.run([_nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
            logs.append(link.stdout + link.stderr)
            procs.append(link)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    failed = any(p.returncode != 0 for p in procs)
    if failed or verbose:
        sys.stderr.write("".join(logs))
    if failed:
        raise RuntimeError(f"nvcc failed building {os.path.basename(path)}")
    os.replace(tmp, path)
    return path


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--trace", action="store_true", help="build lib/libb200attn_trace.so (-DATTN_TRACE)")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, trace=a.trace))
