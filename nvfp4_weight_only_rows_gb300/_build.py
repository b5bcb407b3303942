"""Compile the CUDA sources of this package into libnvfp4_lm_head.so (sm_103a).

Each translation unit is compiled by nvcc in parallel, then linked into one
shared library next to this file.  The library links the CUDA runtime
dynamically, so inside a PyTorch process it shares torch's runtime instance.
calls.cpp, the Python side of some calls, is compiled beside them against the
installed torch's headers into _calls.so, which links that library.  A C
caller who has no torch runs this file, which builds the library alone.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libnvfp4_lm_head.so")
CALLS = os.path.join(HERE, "_calls.so")
SOURCES = ("quantize.cu", "lm_head.cu", "fp8.cu", "w4a4.cu", "topk.cu", "api.cu", "noalloc.cu",
           "selftest.cu", "moe_route.cu", "moe.cu", "moe_tc.cu",
           "logprobs.cu")
CALLS_SOURCES = ("calls.cpp",)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build the library")
    return cand


def _stale(sources, target) -> bool:
    """Whether target is older than its sources, a header or this file."""
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f in sources or f.endswith(".cuh")]
    deps += [os.path.join(HERE, "..", "include", "nvfp4_lm_head.h"), __file__]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _torch_id() -> str:
    """What a build of calls.cpp fits: this torch in this Python."""
    import torch

    return f"torch {torch.__version__} at {os.path.dirname(torch.__file__)}, " \
           f"{sysconfig.get_config_var('SOABI')}"


def _calls_stale() -> bool:
    if _stale(CALLS_SOURCES, CALLS):
        return True
    try:
        with open(CALLS + ".for") as f:
            return f.read() != _torch_id()
    except OSError:
        return True


def _compile_calls(obj_dir: str):
    """calls.cpp against the installed torch: (object, link arguments)."""
    import torch

    home = os.path.dirname(torch.__file__)
    obj = os.path.join(obj_dir, "calls.o")
    inc = [os.path.join(home, "include"),
           os.path.join(home, "include", "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    cmd = ["g++", "-O2", "-fPIC", "-std=c++17", "-Wall", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-isystem{p}" for p in inc], "-c", os.path.join(CSRC, "calls.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on calls.cpp:\n{r.stderr}")
    return obj, ["-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """libnvfp4_lm_head.so alone: nvcc, no torch."""
    if not force and not _stale(SOURCES, LIB):
        return LIB
    obj_dir = os.path.join(HERE, "_build")
    os.makedirs(obj_dir, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(obj_dir, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if ptxas_info:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-cudart=shared", "-o", tmp, *[o for o, _ in results],
           "-Xlinker", "-rpath=/usr/local/cuda/lib64"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """The library, and _calls.so against the installed torch.  A failure of the
    second is raised once the library is in place."""
    obj_dir = os.path.join(HERE, "_build")
    os.makedirs(obj_dir, exist_ok=True)
    with cf.ThreadPoolExecutor(1) as ex:
        calls = ex.submit(lambda: _compile_calls(obj_dir) if force or _calls_stale() else None)
        build_library(force, verbose, ptxas_info)
        compiled = calls.result()
    if compiled is None:
        return LIB
    calls_obj, calls_libs = compiled
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, calls_obj, "-L" + HERE, "-l:" + os.path.basename(LIB),
           "-Wl,-rpath,$ORIGIN", *calls_libs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _calls.so failed:\n{r.stderr}")
    os.replace(tmp, CALLS)
    with open(CALLS + ".for", "w") as f:
        f.write(_torch_id())
    return LIB


if __name__ == "__main__":  # a C caller's build
    print(build_library(force=True, verbose=True, ptxas_info=True))
