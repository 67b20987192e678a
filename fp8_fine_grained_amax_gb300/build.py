"""Build libfp8q.so in-tree with nvcc for sm_103a.

Each .cu file is compiled separately (in parallel) and linked into one shared
library next to this file.  The CUDA runtime is linked statically, and the
driver's tensor-map encoder is looked up at run time, so loading the library
needs no GPU driver (the symbol check in the CPU tests relies on this).

The GEMM kernel gives registers from its control warpgroup to its epilogue
warpgroups with setmaxnreg; that split is only valid if ptxas builds the
kernel for exactly the launch register count the source assumes
(``kLaunchRegs`` in csrc/gemm.cu).  The build reads ptxas' report and refuses
to link a library that breaks this.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfp8q.so")
# The argument marshalling of the newer calls as a CPython module (linked
# against the library and torch).  The other calls need neither it nor torch's
# headers: where it does not build, the library still does.
EXT = os.path.join(PKG, "_torch_calls.so")
EXT_SOURCE = "torch_calls.cpp"
EXT_MADE_FOR = os.path.join(BUILD, "torch_calls.made_for")  # the torch and the interpreter that EXT is linked against
SOURCES = ["gemm.cu", "gemm_mx.cu", "quant.cu", "swiglu.cu", "newton_schulz.cu", "api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin on PATH)")


def _current(target: str, inputs) -> bool:
    """Whether `target` is there and no older than what it is made from."""
    files = [*inputs, os.path.join(INCLUDE, "fp8q.h"), os.path.abspath(__file__)]
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in files)


def _lib_current() -> bool:
    return _current(LIB, [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != EXT_SOURCE])


def _made_for() -> str:
    import torch
    return f"torch {torch.__version__} in {os.path.dirname(torch.__file__)}, python {sys.version}"


def _ext_current() -> bool:
    if not _current(EXT, [os.path.join(CSRC, EXT_SOURCE)]) or not os.path.exists(EXT_MADE_FOR):
        return False
    with open(EXT_MADE_FOR) as f:
        return f.read() == _made_for()


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-Xptxas", "-v", "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _compile_ext() -> str:
    """Object file of the CPython module (torch's headers, host code only)."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    obj = os.path.join(BUILD, "torch_calls.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    inc = [*include_paths(), sysconfig.get_paths()["include"], cuda, INCLUDE]
    cmd = [shutil.which("g++") or "g++", "-O1", "-std=c++17", "-fPIC", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{d}" for d in inc], "-c", os.path.join(CSRC, EXT_SOURCE), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {EXT_SOURCE}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_ext(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libfp8q.so",
           f"-L{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {EXT_SOURCE} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)
    with open(EXT_MADE_FOR, "w") as f:
        f.write(_made_for())


def launch_regs_of(gemm_src: str) -> int:
    """The per-thread launch register count the GEMM source is written for."""
    m = re.search(r"constexpr int kLaunchRegs = (\d+);", open(gemm_src).read())
    if not m:
        raise RuntimeError("kLaunchRegs not found in " + gemm_src)
    return int(m.group(1))


def check_gemm_registers(ptxas_log: str, expected: int, kernel: str = "fp8q_gemm_kernel") -> None:
    """Every instantiation of `kernel` must be built for `expected` registers."""
    entries = re.split(r"Compiling entry function", ptxas_log)
    found = 0
    for e in entries:
        if kernel not in e.split("\n", 1)[0]:
            continue
        m = re.search(r"Used (\d+) registers", e)
        if not m or int(m.group(1)) != expected:
            raise RuntimeError(
                "GEMM kernel not built for %d registers per thread (ptxas: %s); the "
                "setmaxnreg split would not balance" % (expected, m and m.group(0)))
        found += 1
    if found == 0:
        raise RuntimeError("ptxas report names no " + kernel)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile what is stale and return the path of libfp8q.so.  A marshalling
    module that does not build is a warning; its calls raise when they are used."""
    stale_lib, stale_ext = force or not _lib_current(), force or not _ext_current()
    if not (stale_lib or stale_ext):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        ext = ex.submit(_compile_ext) if stale_ext else None
        if stale_lib:
            _link_library(dict(zip(SOURCES, ex.map(_compile, SOURCES))), verbose)
    if ext is not None:
        try:
            _link_ext(ext.result())
        except Exception as e:
            if os.path.exists(EXT):
                os.remove(EXT)  # made from other sources or for another torch
            warnings.warn(f"the marshalling module was not built: {e}", RuntimeWarning, stacklevel=2)
    return LIB


def _link_library(results, verbose: bool) -> None:
    """libfp8q.so from each source's object file and ptxas report."""
    check_gemm_registers(results["gemm.cu"][1], launch_regs_of(os.path.join(CSRC, "gemm.cu")))
    check_gemm_registers(results["gemm_mx.cu"][1], launch_regs_of(os.path.join(CSRC, "gemm_mx.cu")),
                         "fp8q_gemm_mx_kernel")
    check_gemm_registers(results["newton_schulz.cu"][1],
                         launch_regs_of(os.path.join(CSRC, "newton_schulz.cu")), "ns_steps_kernel")
    if verbose:
        for src, (_, log) in results.items():
            print(f"== {src}\n{log}")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-Xlinker", "-soname=libfp8q.so", "-o", tmp,
           *[results[s][0] for s in SOURCES]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build_library(force=True, verbose=True))
