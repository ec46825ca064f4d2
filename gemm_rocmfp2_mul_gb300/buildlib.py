"""Build librfp2.so in-tree with nvcc for sm_103a.

Every ``csrc/*.cu`` file is one translation unit; they are compiled in
parallel and linked into ``_build/librfp2.so`` (git-ignored).
That needs nvcc alone.  Where torch is installed, ``csrc/binding.cpp`` is
compiled beside them against it and linked to that library as
``_build/_rfp2_binding.so``, for that torch and Python alone
(``_build/binding.txt``).  ptxas resource reports (registers, spills, shared
memory) go to ``_build/ptxas.log``.

Run ``python -m gemm_rocmfp2_mul_gb300.buildlib`` or call :func:`build`.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
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


def _newer(built: str, sources) -> bool:
    headers = glob.glob(os.path.join(os.path.dirname(HERE), "include", "*.h"))
    newest = max(os.path.getmtime(f) for f in [*sources, *headers, os.path.abspath(__file__)])
    return os.path.exists(built) and os.path.getmtime(built) >= newest


def _library_up_to_date() -> bool:
    return _newer(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")))


def binding_for() -> str | None:
    """What a binding built here is for; None without torch."""
    if importlib.util.find_spec("torch") is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        import torch
        version = torch.__version__
    return f"torch {version}, {sys.implementation.cache_tag}"


def binding_fits() -> bool:
    """Is the binding that is there for the torch and the Python that run?"""
    stamp = os.path.join(BUILD, "binding.txt")
    if not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        return f.read() == binding_for()


def _binding_up_to_date() -> bool:
    return binding_for() is None or (binding_fits() and _newer(BINDING, [os.path.join(CSRC, "binding.cpp")]))


def up_to_date() -> bool:
    return _library_up_to_date() and _binding_up_to_date()


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
    with open(os.path.join(BUILD, "binding.txt"), "w") as f:
        f.write(binding_for())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link librfp2.so, and the binding where torch is installed; returns the library's path."""
    library = force or not _library_up_to_date()
    binding = binding_for() is not None and (force or not _binding_up_to_date())
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources() if library else []
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding) if binding else None
        results = list(ex.map(_compile, srcs))
    if library:
        tmp = LIB + f".tmp{os.getpid()}"
        _run([_nvcc()] + ARCH + ["-shared", "-Xlinker", "-soname=" + os.path.basename(LIB), "-o", tmp]
             + [obj for obj, _ in results], "link")
        os.replace(tmp, LIB)
        logs = "\n".join(log for _, log in results)
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            f.write(logs)
        if verbose:
            print(logs)
    if binding:
        _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
