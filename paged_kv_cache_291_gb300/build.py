"""Build libpagedkv.so in-tree with nvcc for sm_103a.

Each .cu under csrc/ is compiled to an object in parallel, then the objects
are linked into ``libpagedkv.so`` beside this file (CUDA runtime linked
statically, only the ``pkv_*`` symbols exported).  csrc/binding.cpp, the
CPython module that hands torch tensors to some of the calls, is compiled
against the installed torch at the same time; without a torch, or where that
module does not build, the library is complete all the same.  Used by
``__graft_entry__.build()`` and by the package on import when the library is
stale; it needs nvcc but no GPU.
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
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpagedkv.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libpagedkv needs the CUDA toolkit to build")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files.append(os.path.join(INCLUDE, "pkv.h"))
    files += [BINDING_SRC, os.path.abspath(__file__)]
    return files


def _targets():
    return [LIB, BINDING] if importlib.util.find_spec("torch") is not None else [LIB]


def up_to_date() -> bool:
    if not all(os.path.exists(f) for f in _targets()):
        return False
    t = min(os.path.getmtime(f) for f in _targets())
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
                     "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]
    if ptxas_verbose:
        common += ["-Xptxas", "-v"]
    common += os.environ.get("PKV_NVCC_FLAGS", "").split()  # extra flags for tuning builds

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        cmd = [cc, "-c", src, "-o", obj] + common
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_verbose:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    binding_obj = os.path.join(BUILD, "binding.o")

    def compile_binding():
        import torch
        from torch.utils import cpp_extension
        cmd = [os.environ.get("CXX", "g++"), "-c", BINDING_SRC, "-o", binding_obj, "-O2", "-std=c++17", "-fPIC",
               "-fvisibility=hidden", "-w", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
               "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
               "-I", os.path.join(os.path.dirname(os.path.dirname(cc)), "include")]
        for d in cpp_extension.include_paths():
            cmd += ["-isystem", d]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed on binding.cpp:\n{r.stdout}\n{r.stderr}")

    with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as ex:
        binding = ex.submit(compile_binding) if BINDING in _targets() else None
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, "-shared"] + ARCH + ["-o", tmp] + objs + ["-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if binding is None:
        return LIB
    binding.result()
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, binding_obj, "-L", HERE, "-lpagedkv", "-L", libs,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,$ORIGIN,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv)
    print(LIB)
