"""Builds libmoe_w4a16.so in-tree from csrc/ with nvcc for sm_100a.

    python quantized_mixture_experts_grouped_b200/build.py [--force] [--verbose]

(run by path: importing the package loads the library this script builds)

Each .cu file is compiled to an object under _build/ (in parallel, skipped when up to date),
then linked into a shared library next to this file. The CUDA runtime is linked statically so
the library does not depend on the runtime that torch happens to ship. csrc/binding.cpp, the native
half of the Python binding, becomes the extension module _rows.so (g++, torch's headers), linked
against that library; _rows.so.stamp beside it records the torch and the interpreter it was built for, and
it is built again when they change.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe_w4a16.so")
BINDING = os.path.join(PKG, "_rows.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-I", INCLUDE, "-I", CSRC, "-prec-div=true", "-prec-sqrt=true", "-ftz=false", "-Xptxas", "-warn-spills"]


def _nvcc():
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(cuda, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def _deps():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _compile(src: str, verbose: bool, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    newest = max([os.path.getmtime(src)] + [os.path.getmtime(d) for d in _deps()])
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest and not extra:
        return obj
    cmd = [_nvcc(), *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)
    return obj


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    extra = list(extra or [])
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, extra), srcs))
    if force or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs) or extra:
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [_nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    _build_binding(force, verbose)
    return LIB


def _binding_command(out: str) -> list[str]:
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    return ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
            "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
            "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"), os.path.join(CSRC, "binding.cpp"), "-o", out, "-L", PKG,
            "-l:libmoe_w4a16.so", "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
            "-lc10", "-Wl,-rpath,$ORIGIN"]      # torch's own libraries are loaded by then


def _binding_stamp() -> str:
    """What _rows.so is bound to besides its sources: torch, its C++ ABI, the interpreter, the command."""
    import sysconfig

    import torch
    return "\n".join([torch.__version__, str(torch.version.git_version), str(sysconfig.get_config_var("SOABI")),
                      *_binding_command(BINDING)]).replace(ROOT, ".")      # wherever the tree lies


def _binding_is_current(binding: str = BINDING, stamp: str | None = None) -> bool:
    """Whether `binding` is newer than its sources and was built for this torch and this interpreter."""
    sources = [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "moe_w4a16.h")]
    if not os.path.exists(binding) or any(os.path.getmtime(binding) < os.path.getmtime(s) for s in sources):
        return False
    try:
        with open(binding + ".stamp") as f:
            return f.read() == (_binding_stamp() if stamp is None else stamp)
    except OSError:
        return False


def _build_binding(force: bool, verbose: bool) -> None:
    if not force and _binding_is_current():
        return
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = _binding_command(tmp)
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(BINDING + ".stamp"):      # none stands beside a module it does not describe
        os.remove(BINDING + ".stamp")
    os.replace(tmp, BINDING)
    with open(BINDING + ".stamp", "w") as f:
        f.write(_binding_stamp())


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
