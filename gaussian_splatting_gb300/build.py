"""Build libgs.so in-tree: every csrc/*.cu compiled for sm_103a in parallel, then linked; and _dense.so,
the Python functions of the dense layers over it (csrc/dense_binding.cpp, against PyTorch's headers).

Usage: ``python -m gaussian_splatting_gb300.build`` (or ``build()`` from Python).
The library links the shared CUDA runtime so it shares the process's runtime with
PyTorch.  No fast-math: the kernels rely on IEEE division and square root.
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
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libgs.so")
BINDING = os.path.join(HERE, "_dense.so")
BUILD_DIR = os.path.join(HERE, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
                     "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: set NVCC or install the CUDA toolkit")
    return cand


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _binding_flags() -> tuple[list[str], list[str]]:
    """Compiler and linker flags of _dense.so."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    flags = ["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    flags += [f for i in inc for f in ("-isystem", i)]
    # (PyTorch's libraries are in the process already when the module is imported)
    libs = [f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
            f"-L{HERE}", "-l:libgs.so", "-Wl,-rpath,$ORIGIN"]
    return flags, libs


def _stale() -> bool:
    if not os.path.exists(OUT) or not os.path.exists(BINDING):
        return True
    t = min(os.path.getmtime(OUT), os.path.getmtime(BINDING))
    deps = sources() + [os.path.join(CSRC, "dense_binding.cpp")] + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(HERE, "..", "include", "gs.h")]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile the CUDA sources and the binding, link libgs.so and _dense.so; returns libgs.so's path."""
    if not force and not _stale():
        return OUT
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = NVCC_FLAGS + list(extra_flags or [])
    srcs = sources()

    binding = os.path.join(CSRC, "dense_binding.cpp")
    gxx = shutil.which("g++") or "g++"
    cxx_flags, libs = _binding_flags()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [gxx, *cxx_flags, "-c", src, "-o", obj] if src == binding else [nvcc, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(12, len(srcs) + 1)) as ex:
        *objs, binding_obj = ex.map(compile_one, srcs + [binding])
    tmp = OUT + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OUT)
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [gxx, "-shared", "-o", tmp, binding_obj, *libs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
