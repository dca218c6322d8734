"""Build libgqa_attn.so in-tree with nvcc for sm_103a.

Usage: ``python -m gqa_attention_gb300.build`` (or ``build()`` from Python).
Each ``csrc/*.cu`` is compiled in parallel to an object under ``_build/`` and
the objects are linked into ``gqa_attention_gb300/libgqa_attn.so`` against the
shared CUDA runtime (``libcudart.so.13``), so that a process that also uses
PyTorch holds one runtime instance.  ``csrc/torch_binding.cpp``, the helpers for
torch tensors of the block-scaled cache, is compiled against the installed
PyTorch to ``_torch_binding.so`` at the same time; the library itself needs neither
PyTorch nor Python's headers.  Rebuilds only what changed.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgqa_attn.so")
TORCH_BINDING = os.path.join(PKG, "_torch_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def cuda_home() -> str:
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if home and os.path.exists(os.path.join(home, "bin", "nvcc")):
        return home
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def _nvcc() -> str:
    return os.path.join(cuda_home(), "bin", "nvcc")


def _cflags(extra=()):
    return [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
            "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC, *extra]


def _deps_mtime() -> float:
    files = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str, obj: str, extra) -> str:
    cmd = [_nvcc(), *_cflags(extra), "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}\n{r.stdout}")
    return r.stderr


def build_torch_binding(force: bool = False) -> str:
    """Compile csrc/torch_binding.cpp for the installed Python and PyTorch; return its path."""
    import torch

    src = os.path.join(CSRC, "torch_binding.cpp")
    header = os.path.join(INCLUDE, "gqa_attn.h")
    stamp = os.path.join(BUILD, "torch_binding.stamp")  # what the module was built for
    built_for = f"{sys.version} {torch.__version__}"
    os.makedirs(BUILD, exist_ok=True)
    if not force and os.path.exists(TORCH_BINDING) and os.path.exists(stamp) and \
            open(stamp).read() == built_for and os.path.getmtime(TORCH_BINDING) >= max(
                os.path.getmtime(src), os.path.getmtime(header), os.path.getmtime(__file__)):
        return TORCH_BINDING
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    tmp = TORCH_BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(root, "include"),
           "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(cuda_home(), "include"), "-I" + INCLUDE, src, "-o", tmp,
           "-L" + lib, "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-lc10",
           "-lc10_cuda", "-ldl",
           "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for torch_binding.cpp:\n{r.stderr}\n{r.stdout}")
    os.replace(tmp, TORCH_BINDING)
    with open(stamp, "w") as f:
        f.write(built_for)
    return TORCH_BINDING


def build(force: bool = False, verbose: bool = False, extra_flags=(), lib_path: str = LIB,
          build_dir: str = BUILD) -> str:
    """Compile every csrc/*.cu for sm_103a and link libgqa_attn.so; return its path.

    ``extra_flags``, ``lib_path`` and ``build_dir`` let a tuning run build a
    variant (e.g. ``-DGQA_DECODE_STAGES_D128=4``) beside the default library.
    With the default library the torch binding is built too, where PyTorch is
    installed.  If that fails the library stands all the same and the reason goes to
    stderr: the helpers that need the binding build it again and raise.
    """
    BUILD_, LIB_ = build_dir, lib_path
    os.makedirs(BUILD_, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    dep_t = _deps_mtime()
    jobs = []
    for src in srcs:
        obj = os.path.join(BUILD_, os.path.basename(src)[:-3] + ".o")
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(
                os.path.getmtime(src), dep_t):
            jobs.append((src, obj))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 1))) as ex:
        binding = None
        if os.path.abspath(LIB_) == os.path.abspath(LIB) and importlib.util.find_spec("torch"):
            binding = ex.submit(build_torch_binding, force)
        futs = {ex.submit(_compile, s, o, list(extra_flags)): s for s, o in jobs}
        for f in cf.as_completed(futs):
            msg = f.result()
            if verbose and msg:
                print(f"[{os.path.basename(futs[f])}]\n{msg}", file=sys.stderr)
    objs = [os.path.join(BUILD_, os.path.basename(s)[:-3] + ".o") for s in srcs]
    if jobs or force or not os.path.exists(LIB_):
        lib64 = os.path.join(cuda_home(), "lib64")
        tmp = LIB_ + f".tmp{os.getpid()}"
        cmd = [_nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
               "-Xlinker", f"-rpath,{lib64}", "-Xlinker", "--no-undefined"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}\n{r.stdout}")
        os.replace(tmp, LIB_)
    if binding is not None and binding.exception() is not None:
        print(f"torch binding not built: {binding.exception()}", file=sys.stderr)
    return LIB_


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
    print(LIB)
