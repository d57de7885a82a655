"""Builds libsdp.so in-tree: one nvcc process per translation unit, in
parallel, for sm_103a only, then a shared-library link; and beside it the
serving operators' Python binding (_serving.*.so, C++ against this Python and torch, which its name says).

    python -m gqa_flash_attention_gb300.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

from .serving import BINDING_PATH

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsdp.so")
BINDING_SRC = os.path.join(PKG, "binding", "binding.cpp")

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
         "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]


def _compile(src: str) -> str:
    name = os.path.splitext(os.path.basename(src))[0]
    obj = os.path.join(BUILD, name + ".o")
    log = os.path.join(BUILD, name + ".ptxas.log")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(log, "w") as f:
        f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_binding() -> str:
    """The binding's object file; linked once libsdp.so is there."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    obj = os.path.join(BUILD, "binding.o")
    system = [sysconfig.get_paths()["include"], *cpp_extension.include_paths(), _cuda_include()]  # no warnings from these
    cmd = [os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-Wextra",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
           *(x for i in system for x in ("-isystem", i)), "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {BINDING_SRC} failed:\n{r.stdout}\n{r.stderr}")
    sys.stderr.write(r.stderr)  # warnings
    return obj


def _cuda_include() -> str:
    import shutil
    nvcc = shutil.which(NVCC)
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include") if nvcc else ""


def _link_binding(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libsdp.so", "-Wl,-rpath,$ORIGIN",
           f"-L{lib}", f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {BINDING_PATH} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)


def _is_new(target: str, sources) -> bool:
    return os.path.exists(target) and os.path.getmtime(target) >= max(os.path.getmtime(p) for p in sources)


def build(force: bool = False) -> str:
    """Compile every CUDA source for sm_103a, link gqa_flash_attention_gb300/libsdp.so, and build the binding."""
    os.makedirs(BUILD, exist_ok=True)
    if not force and _is_new(LIB, _deps()):
        if not _is_new(BINDING_PATH, [*_deps(), BINDING_SRC]):
            _link_binding(_compile_binding())
        return LIB
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(2, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, srcs))
        binding_obj = binding.result()
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([NVCC, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding_obj)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv))
