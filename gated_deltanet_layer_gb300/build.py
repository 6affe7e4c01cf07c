"""Build the in-tree CUDA library (libgdn_decode.so) for sm_103a with nvcc, and the
compiled part of the Python binding (_binding.so) with the host's compiler.

Each translation unit under csrc/ compiles in parallel; the objects link into
one shared library next to this file. Nothing is installed anywhere.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgdn_decode.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_ABI = os.path.join(OBJDIR, "binding.abi")  # what _binding.so was built against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE]


def _nvcc() -> str:
    cands = []
    if os.environ.get("CUDA_HOME"):
        cands.append(os.path.join(os.environ["CUDA_HOME"], "bin", "nvcc"))
    cands.append("/usr/local/cuda/bin/nvcc")
    w = shutil.which("nvcc")
    if w:
        cands.append(w)
    for c in cands:
        if os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found (set CUDA_HOME)")


def _cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def _abi() -> str:
    """The torch and the Python that _binding.so belongs to: its C++ ABI is theirs."""
    import torch
    return " ".join((torch.__version__, str(torch.version.git_version), os.path.dirname(torch.__file__), sys.implementation.cache_tag))


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(BINDING) and os.path.exists(BINDING_ABI)):
        return False
    with open(BINDING_ABI) as f:
        if f.read() != _abi():
            return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(d) <= t for d in _deps())


def _build_binding(cuda_home: str) -> None:
    """Against the installed torch's headers, whose libraries the process has loaded by then."""
    import sysconfig

    import torch
    T = os.path.dirname(torch.__file__)
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", os.path.join(CSRC, "gdn_binding.cpp"), "-o", tmp, "-I", INCLUDE]
    for d in (os.path.join(T, "include"), sysconfig.get_paths()["include"], os.path.join(cuda_home, "include")):
        cmd += ["-isystem", d]
    cmd += [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-L", os.path.join(T, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + os.path.join(T, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the binding does not compile:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_ABI, "w") as f:
        f.write(_abi())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every translation unit, link libgdn_decode.so and the binding. Returns the library's path."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OBJDIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, "-c", src, "-o", obj] + ARCH + NVCC_FLAGS + extra
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_build_binding, os.path.dirname(os.path.dirname(nvcc)))
        results = list(ex.map(compile_one, _sources()))
        binding.result()
    if verbose or ptxas_info:
        for _, log in results:
            if log.strip():
                print(log, file=sys.stderr)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-shared", "-o", tmp] + objs + ARCH + [
        "-cudart", "shared", "-Xlinker", "-rpath," + _cuda_lib_dir(nvcc)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
