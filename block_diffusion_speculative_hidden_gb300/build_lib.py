"""Build libdflash.so in-tree with nvcc for sm_103a, and _faces.so beside it.

Usage: python -m block_diffusion_speculative_hidden_gb300.build_lib
Compiles every csrc/*.cu in parallel into _build/ and links the shared
library next to this file.  No CMake, one -gencode.  csrc/faces.cpp, the
compiled Python faces of some of its calls, needs the host compiler and the
headers of Python and PyTorch.
"""
from __future__ import annotations

import concurrent.futures as fut
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(os.path.dirname(PKG), "_build", "libdflash")
LIB = os.path.join(PKG, "libdflash.so")
FACES = os.path.join(PKG, "_faces.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def cuda_lib_dir() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(nvcc())), "lib64")


FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", os.path.join(os.path.dirname(PKG), "include")]


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if (os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(src)
            and all(os.path.getmtime(obj) >= os.path.getmtime(h)
                    for h in glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                    + [os.path.join(os.path.dirname(PKG), "include", "dflash.h")])):
        return obj
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _cxx() -> str:
    return shutil.which("g++") or shutil.which("c++") or "c++"


def _torch_dir() -> str:
    return list(importlib.util.find_spec("torch").submodule_search_locations)[0]


def _compile_faces() -> str:
    src, obj = os.path.join(CSRC, "faces.cpp"), os.path.join(BUILD, "faces.o")
    include = os.path.join(os.path.dirname(PKG), "include")
    # The object is of one PyTorch and one Python, whose files may be older than it: what it was compiled
    # for stands beside it.
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        want = "\n".join([_torch_dir(), f.read(), sys.version, sysconfig.get_paths()["include"]])
    stamp = obj + ".for"
    have = None
    if os.path.exists(stamp):
        with open(stamp) as f:
            have = f.read()
    deps = [src, os.path.join(include, "dflash.h")]
    if os.path.exists(obj) and have == want and all(os.path.getmtime(obj) >= os.path.getmtime(d) for d in deps):
        return obj
    inc = os.path.join(_torch_dir(), "include")
    cmd = [_cxx(), "-std=c++17", "-O2", "-fPIC", "-Wall",
           "-D_GLIBCXX_USE_CXX11_ABI=1"]
    for d in (inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
              os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")):
        cmd += ["-isystem", d]
    r = subprocess.run([*cmd, "-I", include, "-c", src, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {src} failed:\n{r.stdout}\n{r.stderr}")
    with open(stamp, "w") as f:
        f.write(want)
    return obj


def _link_faces(obj: str) -> None:
    if os.path.exists(FACES) and all(os.path.getmtime(FACES) >= os.path.getmtime(o) for o in (obj, LIB)):
        return
    libs = os.path.join(_torch_dir(), "lib")
    cmd = [_cxx(), "-shared", "-o", FACES + ".tmp", obj, "-L", PKG, "-l:libdflash.so",
           "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,$ORIGIN:{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {FACES} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(FACES + ".tmp", FACES)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with fut.ThreadPoolExecutor(max_workers=min(8, len(srcs)) + 1) as ex:
        faces = ex.submit(_compile_faces)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    if os.path.exists(LIB) and not force and all(os.path.getmtime(LIB) >= os.path.getmtime(o) for o in objs):
        _link_faces(faces.result())
        return LIB
    libdir = cuda_lib_dir()
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", LIB + ".tmp", *objs,
           "-L", libdir, "-Xlinker", f"-rpath,{libdir}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(LIB + ".tmp", LIB)
    _link_faces(faces.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
