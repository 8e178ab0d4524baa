"""Builds libdfa.so (the C-ABI attention library) in-tree for sm_103a.

Every translation unit under ``csrc/`` is compiled by nvcc in parallel into
``_build/`` and linked into ``long_context_causal_gb300/libdfa.so`` with the
CUDA runtime linked statically.  Beside it, ``binding/dfa_torch.cpp`` becomes
the extension module ``_dfa_torch`` (host code only, against this torch).  Set ``DFA_PTXAS_VERBOSE=1`` to print
register / shared-memory use per kernel.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
BUILD = os.path.join(os.path.dirname(PKG), "_build")
LIB = os.path.join(PKG, "libdfa.so")
BINDING = os.path.join(PKG, "binding", "dfa_torch.cpp")
BINDING_LIB = os.path.join(PKG, "_dfa_torch.so")
BINDING_KEY = os.path.join(BUILD, "dfa_torch.key")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdfa.so")


def _flags() -> list[str]:
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                "--expt-relaxed-constexpr", "-Xcompiler", "-Wall"]
    if os.environ.get("DFA_PTXAS_VERBOSE"):
        f += ["-Xptxas", "-v"]
    return f


def _sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps() -> list[str]:
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _binding_command(cuda: str) -> list[str]:
    """The host compiler's command against the torch that runs, without the output; cuda: the toolkit's folder."""
    import sysconfig

    import torch
    root = os.path.join(os.path.dirname(torch.__file__))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return (["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] +
            ["-isystem" + i for i in include] + [BINDING, "-L" + os.path.join(root, "lib")] +
            ["-l" + x for x in ("torch_python", "torch", "torch_cpu", "c10", "c10_cuda")])


def _binding_key() -> str:
    """What the module is built against: it fits no other torch or Python.  (The
    toolkit, for whose runtime headers alone it is needed, may be gone since.)"""
    import sys

    import torch
    return "\n".join([f"torch {torch.__version__}", f"python {sys.version}", *_binding_command("")])


def binding_up_to_date() -> bool:
    if not os.path.exists(BINDING_LIB) or not os.path.exists(BINDING_KEY):
        return False
    t = os.path.getmtime(BINDING_LIB)
    if any(os.path.getmtime(d) > t for d in [BINDING] + glob.glob(os.path.join(INCLUDE, "*.h"))):
        return False
    with open(BINDING_KEY) as f:
        return f.read() == _binding_key()


def build_binding() -> str:
    """The extension module, and beside the objects what it was built against."""
    tmp = BINDING_LIB + f".tmp{os.getpid()}"
    r = subprocess.run(_binding_command(os.path.dirname(os.path.dirname(_nvcc()))) + ["-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(BINDING)}:\n{r.stdout}\n{r.stderr}")
    os.makedirs(BUILD, exist_ok=True)
    if os.path.exists(BINDING_KEY):
        os.remove(BINDING_KEY)
    os.replace(tmp, BINDING_LIB)
    with open(BINDING_KEY, "w") as f:
        f.write(_binding_key())
    return BINDING_LIB


def build(force: bool = False, verbose: bool = False) -> str:
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        binding = None if binding_up_to_date() and not force else ex.submit(build_binding)
        build_library(force, verbose)
        if binding:
            binding.result()
    return LIB


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    flags = _flags()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc] + flags + ["-c", src, "-o", obj]
        if src.endswith(".cpp"):
            cmd = [nvcc] + flags + ["-x", "cu", "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose or os.environ.get("DFA_PTXAS_VERBOSE"):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lpthread"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
