"""Build librfp2.so in-tree with nvcc for sm_103a.

Every ``csrc/*.cu`` file is one translation unit; they are compiled in
parallel and linked into ``_build/librfp2.so`` (git-ignored).
``csrc/binding.cpp`` is compiled beside them against the installed torch and
linked to that library as ``_build/_rfp2_binding.so``.  ptxas resource
reports (registers, spills, shared memory) go to ``_build/ptxas.log``.

Run ``python -m gemm_rocmfp2_mul_gb300.buildlib`` or call :func:`build`.
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
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "librfp2.so")
BINDING = os.path.join(BUILD, "_rfp2_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags():
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "-Xptxas", "-v", "--expt-relaxed-constexpr",
                   "-I", os.path.join(os.path.dirname(HERE), "include")]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps_mtime():
    files = _sources() + glob.glob(os.path.join(CSRC, "*.c*h")) + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(
        os.path.join(os.path.dirname(HERE), "include", "*.h")) + [os.path.abspath(__file__)]
    return max(os.path.getmtime(f) for f in files)


def up_to_date() -> bool:
    newest = _deps_mtime()
    return all(os.path.exists(f) and os.path.getmtime(f) >= newest for f in (LIB, BINDING))


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [_nvcc()] + _flags() + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _run(cmd, what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _torch_dir() -> str:
    import torch
    return os.path.dirname(os.path.abspath(torch.__file__))


def _compile_binding() -> str:
    import torch
    obj = os.path.join(BUILD, "binding.o")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [os.path.join(_torch_dir(), "include"), os.path.join(cuda, "include"),
               sysconfig.get_paths()["include"]]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
          *(a for d in include for a in ("-isystem", d)), "-I", os.path.join(os.path.dirname(HERE), "include"),
          "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj], "g++ for binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    tmp = BINDING + f".tmp{os.getpid()}"
    lib = os.path.join(_torch_dir(), "lib")
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
          "-L" + BUILD, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib], "linking the binding")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link librfp2.so; returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    logs = []
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(_compile, srcs))
        binding = binding.result()
    objs = [o for o, _ in results]
    logs = [l for _, l in results]
    tmp = LIB + f".tmp{os.getpid()}"
    _run([_nvcc()] + ARCH + ["-shared", "-Xlinker", "-soname=" + os.path.basename(LIB), "-o", tmp] + objs, "link")
    os.replace(tmp, LIB)
    _link_binding(binding)
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        f.write("\n".join(logs))
    if verbose:
        print("\n".join(logs))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
