"""Builds libattn_gb300.so in place from csrc/*.cu with nvcc for sm_103a, and _native.so, the
marshalling of the calls that last a few microseconds, from csrc/native.cpp with the host compiler.

Each translation unit compiles in its own process (in parallel), then
one link step produces the shared library next to this file.  The CUDA
runtime is linked statically, so loading the library needs no GPU driver;
the driver is reached at run time through the runtime's entry-point query.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libattn_gb300.so")
NATIVE = os.path.join(HERE, "_native.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--threads", "2"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libattn_gb300.so")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newer(than: str) -> bool:
    """Whether the file is missing or older than a source."""
    if not os.path.exists(than):
        return True
    t = os.path.getmtime(than)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps += [os.path.join(HERE, "..", "include", f)
             for f in os.listdir(os.path.join(HERE, "..", "include"))]
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps)


def _torch() -> str:
    """The torch that _native.so is bound to ("": there is none with CUDA)."""
    try:
        import torch
    except ImportError:
        return ""
    return f"{torch.__version__} {os.path.dirname(torch.__file__)} {sys.version}" if torch.version.cuda else ""


def _built_for() -> str:
    try:
        with open(os.path.join(BUILD, "native.torch")) as f:
            return f.read()
    except OSError:
        return ""


def _native() -> None:
    """_native.so against the torch that imports it."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = NATIVE + ".tmp"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
           *(a for i in include for a in ("-isystem", i)), os.path.join(CSRC, "native.cpp"), "-o", tmp,
           "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for native.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)
    with open(os.path.join(BUILD, "native.torch"), "w") as f:
        f.write(_torch())


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False) -> str:
    """Compile and link what changed; returns the library path.

    The library is linked whatever becomes of _native.so, which a torch without CUDA cannot have."""
    against = _torch()
    module = against != "" and (force or _newer(NATIVE) or _built_for() != against)
    library = force or _newer(LIB)
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_v else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-I", CSRC, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_v:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        native = ex.submit(_native) if module else None
        if library:
            objs = list(ex.map(compile_one, sources()))
            tmp = LIB + ".tmp"
            cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, LIB)
        if native is not None:
            native.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_v="--ptxas-v" in sys.argv))
