"""Builds libzc.so in-tree for sm_103a with nvcc (one process per translation unit), and with the host compiler the
Python extension of the operators that take torch tensors natively."""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import fcntl
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libzc.so")
# AddressSanitizer + UndefinedBehaviorSanitizer build of the host code (device
# code is unchanged), for running the CPU-side tests under the sanitizers.
SAN_BUILD = os.path.join(BUILD, "san")
SAN_LIB = os.path.join(LIBDIR, "libzc_san.so")
SAN_FLAGS = ["-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-g"]
SOURCES = ["zc_api.cu", "zc_encode.cu", "zc_decode.cu", "zc_reduce.cu", "zc_hist.cu", "zc_noalloc.cu", "zc_pipeline.cu", "zq.cu",
           "zc_moe.cu", "zc_norm.cu", "zc_norm_bwd.cu"]
TORCH_SOURCE = "zc_torch.cpp"  # the extension, built against the torch at hand
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libzc needs the CUDA toolkit to build")


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "zc.h"), __file__]
    return max(os.path.getmtime(f) for f in files)


def _fresh(target: str) -> bool:
    return os.path.exists(target) and os.path.getmtime(target) >= _deps_mtime()


@contextlib.contextmanager
def _builder_of(target: str):
    """Held while a target is built: of several ranks that find it stale one builds (objects lie in one place), the
    others wait and look again.  The lock goes with its process."""
    os.makedirs(os.path.dirname(target), exist_ok=True)
    with open(target + ".lock", "w") as f:
        fcntl.flock(f, fcntl.LOCK_EX)
        yield


def _compile(src: str, extra: list[str], outdir: str = BUILD) -> str:
    obj = os.path.join(outdir, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc()] + NVCC_FLAGS + extra + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False, sanitize: bool = False) -> str:
    """Compile every translation unit in parallel and link libzc.so; skip if up to date.

    sanitize=True builds libzc_san.so instead: the same library with its host
    code instrumented by AddressSanitizer and UndefinedBehaviorSanitizer.  A
    process that loads it must load the ASan runtime first (LD_PRELOAD)."""
    lib, outdir = (SAN_LIB, SAN_BUILD) if sanitize else (LIB, BUILD)
    if not force and _fresh(lib):
        return lib
    with _builder_of(lib):
        if not force and _fresh(lib):
            return lib
        os.makedirs(outdir, exist_ok=True)
        extra = ["-Xptxas", "-v"] if verbose_ptxas else []
        host = [f for flag in SAN_FLAGS for f in ("-Xcompiler", flag)] if sanitize else []
        with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
            objs = list(ex.map(lambda s: _compile(s, extra + host, outdir), SOURCES))
        tmp = lib + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + host + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    return lib


def torch_extension_path() -> str:
    """The extension is good for one torch, one Python and one kind of machine; its name says which."""
    import sysconfig

    import torch
    return os.path.join(LIBDIR, f"_zc_torch-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _compile_extension() -> str:
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "zc_torch.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], cuda, INCLUDE]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [f for d in inc for f in ("-isystem" if d != INCLUDE else "-I", d)]
    r = subprocess.run(cmd + ["-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the host compiler failed on {TORCH_SOURCE}:\n{r.stdout}\n{r.stderr}")
    return obj


def build_extension(force: bool = False) -> str:
    """Compile and link the torch extension against libzc.so, which is built beside it if stale; skip if up to date."""
    import torch
    path = torch_extension_path()
    if not force and _fresh(path) and _fresh(LIB):
        return path
    with _builder_of(path):
        if not force and _fresh(path) and _fresh(LIB):
            return path
        os.makedirs(BUILD, exist_ok=True)
        with cf.ThreadPoolExecutor(max_workers=1) as ex:
            compiled = ex.submit(_compile_extension)
            build()
            obj = compiled.result()
        lib = os.path.join(os.path.dirname(torch.__file__), "lib")
        tmp = path + f".tmp{os.getpid()}"
        cmd = ["g++", "-shared", "-o", tmp, obj, "-L", LIBDIR, "-lzc", "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu",
               "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link of the torch extension failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, path)
    return path


def build_all() -> None:
    """libzc.so and the torch extension, compiled side by side."""
    build_extension()


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv, sanitize="--sanitize" in sys.argv))
