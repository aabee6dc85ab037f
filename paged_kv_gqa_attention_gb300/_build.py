"""Builds libqa.so in-tree with nvcc for sm_103a (no cmake, no torch
extension machinery): every .cu under csrc/ is compiled in parallel, then
linked into one shared library that exports only the qa_* symbols.  Beside
it the Python binding of the calls whose host time counts (csrc/binding.cpp,
against torch's headers) becomes the module _binding."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libqa.so")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler",
              "-fPIC,-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found; the CUDA 13 toolkit is required to build libqa")
    return exe


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile and link libqa.so, then the Python binding; returns the
    library's path.  Skips what is newer than every source and header.  The
    library needs nvcc alone: without torch, g++ or Python's headers it is
    there all the same, and the error is the binding's."""
    newest = _deps_mtime()
    lib_done, binding_done = (not force and not extra_flags and os.path.exists(f) and os.path.getmtime(f) >= newest
                              for f in (LIB, BINDING))
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:  # beside nvcc's
        binding = None if lib_done and binding_done else ex.submit(_compile_binding)
        if not lib_done:
            _build_library(verbose, extra_flags)
        if binding is not None:
            _link_binding(binding.result())
    return LIB


def _build_library(verbose: bool, extra_flags: list[str] | None) -> None:
    exe = nvcc()
    flags = NVCC_FLAGS + (extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [exe, *ARCH, *flags, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{res.stdout}\n{res.stderr}")
        if verbose and (res.stdout or res.stderr):
            print(res.stdout, res.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [exe, *ARCH, "-shared", "-o", tmp, *objs, "-Xlinker", "--exclude-libs,ALL"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)


def _torch_dir() -> str:
    import importlib.util

    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("the Python binding needs torch's headers and libraries, and torch is not installed")
    return os.path.dirname(spec.origin)


def _run(cmd: list[str], what: str) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stdout}\n{res.stderr}")


def _compile_binding() -> str:
    torch_dir, obj = _torch_dir(), os.path.join(BUILD, "binding.o")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE,
          "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(torch_dir, "include"),
          "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
          "-isystem", os.path.join(cuda, "include"), "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj],
         "g++ on binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    torch_lib, tmp = os.path.join(_torch_dir(), "lib"), BINDING + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-lqa", "-Wl,-rpath,$ORIGIN", "-L", torch_lib, "-ltorch_python",
          "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"], "link of _binding.so")
    os.replace(tmp, BINDING)


if __name__ == "__main__":
    print(build(force=True, verbose=True))
