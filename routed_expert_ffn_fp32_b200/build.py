"""Build the CUDA library in-tree: routed_expert_ffn_fp32_b200/libmoe_b200.so,
and _fp8_binding.so, the argument marshalling of the 8-bit operators' binding.

nvcc -gencode arch=compute_100a,code=sm_100a (B200 only), one object per
csrc/*.cu, linked into a shared library that exports the C ABI of
include/moe.h.  Objects are rebuilt when a source or header is newer.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_b200.so")
BINDING_SRC = os.path.join(CSRC, "moe_fp8_binding.cpp")
BINDING = os.path.join(PKG, "_fp8_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVFLAGS = ["-O3", "-lineinfo", "-std=c++20", "--expt-relaxed-constexpr",
           "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
           "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_b200.so")
    return cand


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_cmd(out: str):
    import sysconfig

    import torch

    home = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    dirs = [INCLUDE, os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
            cuda, sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f for d in dirs for f in ("-isystem", d)], BINDING_SRC, "-o", out, "-L", os.path.join(home, "lib"),
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]


def _binding_env() -> str:
    """What a built binding fits, beside its sources."""
    import torch

    return f"torch {torch.__version__}, Python {sys.version}"


def _binding_stamp() -> str:
    return os.path.join(BUILD, "_fp8_binding.env")


def _binding_stale() -> bool:
    if _stale(BINDING, [BINDING_SRC, __file__, os.path.join(INCLUDE, "moe.h")]):
        return True
    try:
        with open(_binding_stamp()) as f:
            return f.read() != _binding_env()
    except OSError:
        return True


def build(verbose: bool = False, extra_flags=None) -> str:
    """Compile (incrementally) and return the path of the shared library."""
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    headers = _headers()
    flags = NVFLAGS + list(extra_flags or [])
    jobs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if _stale(obj, [src, __file__] + headers):
            jobs.append([nvcc, *ARCH, *flags, "-c", src, "-o", obj])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        log = os.path.join(BUILD, os.path.basename(cmd[cmd.index("-o") + 1]) + ".log")
        with open(log, "w") as f:
            f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({cmd[cmd.index('-o') - 1]}):\n{r.stderr[-6000:]}")
        return r.stderr

    def binding():
        env = _binding_env()
        out = run(_binding_cmd(BINDING))
        with open(_binding_stamp(), "w") as f:
            f.write(env)
        return out

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        beside = ex.submit(binding) if _binding_stale() else None
        for out in ex.map(run, jobs):
            if verbose:
                sys.stderr.write(out)
    if jobs or _stale(LIB, objs):
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB, *objs, "-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
    # last: the library and its C ABI need neither torch's headers nor Python's
    if beside is not None:
        try:
            out = beside.result()
        except Exception as e:
            raise RuntimeError(f"{LIB} is built, the Python binding of its 8-bit operators is not: {e}") from e
        if verbose:
            sys.stderr.write(out)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
