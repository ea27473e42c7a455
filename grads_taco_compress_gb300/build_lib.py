"""Build libtaco.so in-tree with nvcc for sm_103a, and the compiled binding.

``python -m grads_taco_compress_gb300.build_lib`` or ``build()`` compiles every
``csrc/*.cu`` translation unit in parallel and links the shared library into
``grads_taco_compress_gb300/lib/``; beside it goes ``_fp8_binding.so``, the
Python module of csrc/fp8_binding.cpp (host code against torch's headers).
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import pathlib
import shutil
import subprocess
import sysconfig

PKG = pathlib.Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
OUT_DIR = PKG / "lib"
BUILD_DIR = PKG / "_build"
LIB = OUT_DIR / "libtaco.so"
BINDING = OUT_DIR / "_fp8_binding.so"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
          "-I", str(ROOT / "include"), "-I", str(CSRC)]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libtaco")
    return cand


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _compile_binding() -> pathlib.Path:
    """csrc/fp8_binding.cpp -> an object file."""
    import torch
    inc = pathlib.Path(torch.__file__).resolve().parent / "include"
    cuda = pathlib.Path(_nvcc()).resolve().parent.parent / "include"
    obj = BUILD_DIR / "fp8_binding.o"
    dirs = [inc, inc / "torch" / "csrc" / "api" / "include", cuda, sysconfig.get_paths()["include"]]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", str(ROOT / "include"),
          *(a for d in dirs for a in ("-isystem", str(d))), "-c", str(CSRC / "fp8_binding.cpp"), "-o", str(obj)])
    return obj


def _link_binding(obj: pathlib.Path) -> None:
    import torch
    libs = pathlib.Path(torch.__file__).resolve().parent / "lib"
    tmp = OUT_DIR / "_fp8_binding.so.tmp"
    _run(["g++", "-shared", "-o", str(tmp), str(obj), "-L", str(OUT_DIR), "-l:libtaco.so", "-L", str(libs),
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,$ORIGIN,-rpath,{libs}"])
    os.replace(tmp, BINDING)


def build(verbose: bool = False, extra_flags: list[str] | None = None) -> pathlib.Path:
    """Compile and link; returns the library path."""
    nvcc = _nvcc()
    BUILD_DIR.mkdir(exist_ok=True)
    OUT_DIR.mkdir(exist_ok=True)
    sources = sorted(CSRC.glob("*.cu"))
    flags = CFLAGS + (extra_flags or [])
    if verbose:
        flags = flags + ["-Xptxas", "-v"]

    def compile_one(src: pathlib.Path):
        obj = BUILD_DIR / (src.stem + ".o")
        return _run([nvcc, *ARCH, *flags, "-c", str(src), "-o", str(obj)])

    # the slowest to compile first
    sources.sort(key=lambda s: -s.stat().st_size * (2 if s.stem == "fp8_norm" else 1))
    with cf.ThreadPoolExecutor(max_workers=min(len(sources) + 1, max(8, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_compile_binding)
        logs = list(ex.map(compile_one, sources))
        binding_obj = binding.result()
    objs = [str(BUILD_DIR / (s.stem + ".o")) for s in sources]
    tmp = OUT_DIR / "libtaco.so.tmp"
    _run([nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", str(tmp), *objs,
          "-Xlinker", "-rpath,/usr/local/cuda/lib64"])
    os.replace(tmp, LIB)
    _link_binding(binding_obj)
    if verbose:
        print("".join(logs))
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose="-v" in sys.argv))
