"""Build of the CUDA library libkvpaged.so (sm_103a only) and of its native binding _calls.so.

Each translation unit is compiled by nvcc in parallel into _build/, then the
objects are linked into a shared library next to this file.  The CUDA runtime
is linked statically; the driver is reached through the runtime's entry-point
query, so the library loads on machines without a GPU driver (it then reports
KV_ERR_CUDA on any device call).
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkvpaged.so")
BINDING_SRC = os.path.join(PKG, "binding", "calls.cpp")
BINDING = os.path.join(PKG, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I" + INCLUDE,
              "-I" + CSRC, "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(cuda, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _headers() -> list[str]:
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _deps() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + _headers()


def _newer(target: str, deps: list[str]) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def _binding_abi() -> str:
    """What the binding is compiled against beside the library: another torch or Python may lay its
    objects out differently, whatever the files' times."""
    import torch
    return f"torch {torch.__version__} at {os.path.dirname(torch.__file__)}, python {sys.version}\n"


def library_up_to_date() -> bool:
    return _newer(LIB, _deps())


def binding_up_to_date() -> bool:
    stamp = os.path.join(BUILD, "binding.abi")
    if not os.path.exists(stamp) or not _newer(BINDING, [BINDING_SRC, *_headers()]):
        return False
    with open(stamp) as f:
        return f.read() == _binding_abi()


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _run(cmd: list[str], what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _build_library(verbose: bool, ptxas_info: bool) -> None:
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        said = _run(cmd, f"nvcc on {os.path.basename(src)}")
        if verbose or ptxas_info:
            sys.stderr.write(said)
        return obj

    # the longest translation units first
    srcs = sorted(sources(), key=lambda f: ("span" not in f, f))
    with ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc, *ARCH, "-shared", "-Xlinker", "-soname=libkvpaged.so", "-o", tmp, *objs], "link")
    os.replace(tmp, LIB)


def _compile_binding() -> tuple[str, str]:
    import torch
    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "binding.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I" + INCLUDE, "-I" + os.path.join(root, "include"),
          "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"),
          "-I" + sysconfig.get_paths()["include"], "-c", BINDING_SRC, "-o", obj], "g++ on calls.cpp")
    return obj, os.path.join(root, "lib")


def _link_binding(obj: str, torch_lib: str) -> None:
    tmp = BINDING + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, LIB, "-L" + torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
          "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib], "link of the binding")
    os.replace(tmp, BINDING)
    with open(os.path.join(BUILD, "binding.abi"), "w") as f:
        f.write(_binding_abi())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link the library and the binding, each where it is not up to date; returns the
    library's path.  The library does not need the binding: where only the binding fails (it wants
    Python's and torch's headers beside g++), the library is in place when the error is raised."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_compile_binding) if force or not binding_up_to_date() else None
        if force or not library_up_to_date():
            _build_library(verbose, ptxas_info)
        if binding is not None:
            _link_binding(*binding.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="-v" in sys.argv))
