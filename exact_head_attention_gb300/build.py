"""Builds libexattn.so in-tree: nvcc for sm_103a, one object per translation
unit (compiled in parallel), static CUDA runtime, no libcuda link (the tensor-map
encoder is fetched through the runtime's driver entry-point query).  Beside it
_binding.so, the Python calls that are marshalled in compiled code: the host
compiler, against the installed torch and libexattn.so."""
from __future__ import annotations

import concurrent.futures
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libexattn.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING_STAMP = os.path.join(BUILD, "binding.torch")  # the torch that it was built against
SOURCES = ["api.cu", "attn_fwd.cu", "fwd_schedule.cu", "attn_bwd.cu", "attn_bwd_dq.cu", "attn_splitkv.cu", "attn_kl.cu", "attn_kl_bwd.cu", "noalloc.cu",
           "cache_api.cu", "cache_io.cu", "cache_attn.cu", "cache_tile.cu", "cache_attn_tree.cu", "cache_tile_tree.cu", "draft_tree.cu", "rope_api.cu", "rope.cu", "cache_append.cu"]
HEADERS = ["ptx.cuh", "kernels.h", "softmax.cuh", "ds_ops.cuh", "kv_order.cuh", "fwd_schedule.h", "fwd_tile.cuh",
           "api_internal.h", "cache.h", "cache8.cuh", "cache_sched.cuh", "cache_attn.cuh", "cache_tile.cuh", "rope.h", "rope.cuh", "cache_io.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
    f"-I{os.path.join(ROOT, 'include')}",
]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _newest_input() -> float:
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(ROOT, "include", "exattn.h"),
                                                                 os.path.abspath(__file__)]
    return max(os.path.getmtime(f) for f in files)


def _torch_stamp() -> str:
    return importlib.metadata.version("torch") + " " + sysconfig.get_python_version()


def _binding_current() -> bool:
    if not (os.path.exists(BINDING) and os.path.exists(BINDING_STAMP)):
        return False
    newest = max(os.path.getmtime(f) for f in (BINDING_SOURCE, os.path.join(ROOT, "include", "exattn.h"), os.path.abspath(__file__)))
    with open(BINDING_STAMP) as f:
        return os.path.getmtime(BINDING) >= newest and f.read() == _torch_stamp()


def _run(cmd, what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _binding_object() -> str:
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    obj = os.path.join(BUILD, "binding.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", *(f"-I{d}" for d in include), "-c", BINDING_SOURCE, "-o", obj], "g++ for binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    torch_lib = os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libexattn.so", "-Wl,-rpath,$ORIGIN", f"-L{torch_lib}", "-lc10", "-ltorch_cpu",
          "-lc10_cuda", "-ltorch_python"], "linking _binding.so")
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(_torch_stamp())


def build(force: bool = False, verbose: bool = False) -> str:
    lib_current = not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input()
    binding_current = not force and _binding_current()
    if lib_current and binding_current:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        said = _run(cmd, f"nvcc for {src}")
        if verbose:
            print(said)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = None if binding_current else ex.submit(_binding_object)
        if not lib_current:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB + f".tmp{os.getpid()}"
            _run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-cudart", "static", "-o", tmp, *objs], "linking libexattn.so")
            os.replace(tmp, LIB)
        if binding is not None:
            _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
