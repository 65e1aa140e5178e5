"""Builds libb2b.so in-tree with nvcc for sm_103a (and nothing else), and the Python binding of
its per-token entry points with g++.

    python -m gemm_conv_chains_gb300.build [--force]

Each .cu file under csrc/ is compiled in parallel to an object under _build/, then linked
into gemm_conv_chains_gb300/libb2b.so.  The library links the shared CUDA runtime, so a
process that already loaded libcudart (e.g. through torch) uses that same instance.
csrc/binding.cpp becomes gemm_conv_chains_gb300/_binding.so, a CPython extension against the
installed torch's headers that calls libb2b.so beside it; another torch or Python has it built anew.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libb2b.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(HERE, "_binding.so")
BINDING_FOR = os.path.join(BUILD_DIR, "binding.for")     # the torch and Python it was compiled against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _cuda_home() -> str:
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if home and os.path.isdir(home):
        return home
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def _nvcc() -> str:
    return shutil.which("nvcc") or os.path.join(_cuda_home(), "bin", "nvcc")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + [os.path.join(INCLUDE, "b2b.h"), BINDING_SRC, os.path.abspath(__file__)]


def _newer_than_sources(path) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _binding_target() -> str:
    import torch
    return f"torch {torch.__version__} in {_torch_dir()}, {sysconfig.get_config_var('SOABI')}"


def _binding_fits() -> bool:
    if not os.path.exists(BINDING_FOR):
        return False
    with open(BINDING_FOR) as f:
        return f.read() == _binding_target()


def up_to_date() -> bool:
    return _newer_than_sources(LIB_PATH) and _newer_than_sources(BINDING_PATH) and _binding_fits()


def compile_flags(extra=()):
    return ["-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC",
            "-Xcompiler", "-Wall", f"-I{INCLUDE}", f"-I{CSRC}", *extra]


def _torch_dir() -> str:
    import torch
    return os.path.dirname(os.path.abspath(torch.__file__))


def _compile_binding() -> str:
    obj = os.path.join(BUILD_DIR, "binding.o")
    inc = os.path.join(_torch_dir(), "include")
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-Wall", f"-I{INCLUDE}", f"-isystem{inc}",
           f"-isystem{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}",
           f"-isystem{os.path.join(_cuda_home(), 'include')}",
           f"-isystem{sysconfig.get_paths()['include']}", "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    libs = os.path.join(_torch_dir(), "lib")
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", obj, "-o", tmp, f"-L{HERE}", "-l:libb2b.so", f"-L{libs}",
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN",
           f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_FOR, "w") as f:
        f.write(_binding_target())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every csrc/*.cu and link libb2b.so and the binding; returns the library path."""
    if not force and not extra_flags and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    if not force and not extra_flags and _newer_than_sources(LIB_PATH):     # another torch or Python
        _link_binding(_compile_binding())
        return LIB_PATH
    nvcc = _nvcc()
    flags = compile_flags(extra_flags)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{' '.join(cmd)}\n"
                               f"{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(compile_one, sources()))
        binding_obj = binding.result()
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    lib64 = os.path.join(_cuda_home(), "lib64")
    cmd = [nvcc, "-shared", *ARCH, "-cudart", "shared", *objs, "-o", tmp,
           "-Xlinker", f"-rpath,{lib64}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    _link_binding(binding_obj)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
