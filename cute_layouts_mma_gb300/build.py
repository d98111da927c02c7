"""Build the CUDA library in-tree: csrc/*.cu -> _build/libtn_gemm.so (sm_103a only).

Each translation unit is compiled in parallel with nvcc, then linked with the
static CUDA runtime.  Re-running is cheap: nothing is rebuilt when no source
or header is newer than the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libtn_gemm.so")
# Test-only variants.  timeout_inject: one pipeline arrival is withheld so that a
# bounded wait runs out (exercises the abandon path).  scale_copy: the block-scaled
# instances move their scales with tcgen05.cp instead of tcgen05.st (the pages' copy
# instruction, kept as a tested compile-time alternative).
VARIANTS = {"timeout_inject": ["-DTN_TIMEOUT_INJECT"], "scale_copy": ["-DTN_SCALE_COPY"]}

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def lib_path(variant: str = "") -> str:
    if not variant:
        return LIB
    return os.path.join(BUILD, variant, f"libtn_gemm_{variant}.so")


def up_to_date(variant: str = "") -> bool:
    lib = lib_path(variant)
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in _deps())


# Instances of the block-scaled FP8 kernel whose promotion warps hold 128 sums a thread (256
# columns over two groups of four warps): they share out the registers that the launch holds,
# so the compiler must have given each thread these (Fp8Config::kRegsLaunch).
SPLIT_REGS = 168
_SPLIT = re.compile(r"Compiling entry function '(\w*gemm_fp8_block_kernel\w*Fp8ConfigILi\d+ELi\d+ELi256E(?:Li\d+E){3}Li8E\w*)'"
                    r".*?Used (\d+) registers", re.S)


def check_register_split(log: str) -> int:
    """Number of register-splitting instances in a compiler log (-Xptxas -v); raises if one of
    them has another register count than its split needs, as every launch of it would be refused."""
    found = _SPLIT.findall(log)
    for name, regs in found:
        if int(regs) != SPLIT_REGS:
            raise RuntimeError(f"{name}: {regs} registers, its split of them needs {SPLIT_REGS}")
    return len(found)


def build(force: bool = False, verbose: bool = False, variant: str = "") -> str:
    """Build the library (variant "" is the product; others are test builds)."""
    lib = lib_path(variant)
    if not force and up_to_date(variant):
        return lib
    outdir = os.path.dirname(lib)
    os.makedirs(outdir, exist_ok=True)
    nvcc = _nvcc()
    extra = VARIANTS[variant] if variant else []

    def compile_one(src):
        obj = os.path.join(outdir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if os.path.basename(src) == "gemm_fp8_block.cu" and check_register_split(r.stderr) == 0:
            raise RuntimeError(f"no register counts in the compiler's log of {src}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(_sources())) as ex:
        results = list(ex.map(compile_one, _sources()))
    if verbose:
        for obj, log in results:
            sys.stderr.write(f"--- {os.path.basename(obj)}\n{log}")
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(BUILD, "_experts_binding.so")


def build_binding(force: bool = False) -> str:
    """Build the compiled Python binding of the expert-layer calls (host code alone)."""
    import sysconfig

    import torch
    stamp = BINDING + ".torch"  # the binding is of one torch version
    key = f"{torch.__version__} {sys.version_info[:2]}"
    deps = [BINDING_SRC, os.path.join(INCLUDE, "tn_experts.h"), os.path.join(INCLUDE, "tn_gemm.h"), os.path.abspath(__file__)]
    if not force and os.path.exists(BINDING) and os.path.exists(stamp) and open(stamp).read() == key and \
            all(os.path.getmtime(d) <= os.path.getmtime(BINDING) for d in deps):
        return BINDING
    os.makedirs(BUILD, exist_ok=True)
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc())) if os.path.sep in _nvcc() else "/usr/local/cuda"
    tmp = f"{BINDING}.tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + os.path.join(home, "include"), "-I" + os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"), "-I" + INCLUDE, BINDING_SRC, "-o", tmp,
           "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-Wl,-rpath," + os.path.join(home, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(stamp + f".tmp{os.getpid()}", "w") as f:
        f.write(key)
    os.replace(stamp + f".tmp{os.getpid()}", stamp)
    return BINDING


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
