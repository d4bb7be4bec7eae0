"""Build the CUDA libraries in-tree: rotated_w4a4_quantized_b200/libconvrot.so
(the W4A4 layer, include/convrot.h), libconvrot_w4a16.so (the W4A16
variant, include/convrot_w4a16.h), libconvrot_nvfp4.so (the NVFP4
variant, include/convrot_nvfp4.h), libconvrot_w4g.so (the group-scaled
few-token variant, include/convrot_w4g.h) and libconvrot_kv4.so (the INT4
cache of keys and values, include/convrot_kv4.h); and the extension module
_decoding (csrc/binding.cpp), the native part of the last two's binding.

    python -m rotated_w4a4_quantized_b200.build [--verbose]

Each library is one translation unit (csrc/convrot.cu, csrc/w4a16.cu,
csrc/nvfp4.cu, csrc/w4g.cu, csrc/kv4.cu)
compiled for sm_100a only, with IEEE
fp32 semantics (no fast-math: the epilogue and the quantiser rely on
correctly rounded multiply, add and divide).  The CUDA runtime is linked
statically; the driver's tensor-map encoder is looked up at run time, so no
link against libcuda is needed and the build runs on a machine without a GPU.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
_INC = os.path.join(os.path.dirname(HERE), "include")
SRC = os.path.join(HERE, "csrc", "convrot.cu")
DEPS = [os.path.join(HERE, "csrc", f) for f in ("convrot.cu", "gemm.cuh", "prep.cuh", "ptx.cuh",
                                                     "skinny.cuh", "decode.cuh")]
HEADER = os.path.join(_INC, "convrot.h")
LIB = os.path.join(HERE, "libconvrot.so")
SRC_W4A16 = os.path.join(HERE, "csrc", "w4a16.cu")
DEPS_W4A16 = [os.path.join(HERE, "csrc", f) for f in ("w4a16.cu", "prep.cuh", "ptx.cuh")] + [
    HEADER, os.path.join(_INC, "convrot_w4a16.h")]
LIB_W4A16 = os.path.join(HERE, "libconvrot_w4a16.so")
SRC_NVFP4 = os.path.join(HERE, "csrc", "nvfp4.cu")
DEPS_NVFP4 = [os.path.join(HERE, "csrc", f) for f in ("nvfp4.cu", "prep.cuh", "ptx.cuh")] + [
    HEADER, os.path.join(_INC, "convrot_nvfp4.h")]
LIB_NVFP4 = os.path.join(HERE, "libconvrot_nvfp4.so")
_SHARED = [os.path.join(HERE, "csrc", f) for f in ("frag.cuh", "host.cuh", "prep.cuh", "ptx.cuh")] + [HEADER]
SRC_W4G = os.path.join(HERE, "csrc", "w4g.cu")
DEPS_W4G = [SRC_W4G, os.path.join(_INC, "convrot_w4g.h")] + _SHARED
LIB_W4G = os.path.join(HERE, "libconvrot_w4g.so")
SRC_KV4 = os.path.join(HERE, "csrc", "kv4.cu")
DEPS_KV4 = [SRC_KV4, os.path.join(_INC, "convrot_kv4.h")] + _SHARED
LIB_KV4 = os.path.join(HERE, "libconvrot_kv4.so")

SRC_BINDING = os.path.join(HERE, "csrc", "binding.cpp")
DEPS_BINDING = [SRC_BINDING, HEADER, os.path.join(_INC, "convrot_w4g.h"), os.path.join(_INC, "convrot_kv4.h")]
LIB_BINDING = os.path.join(HERE, "_decoding" + sysconfig.get_config_var("EXT_SUFFIX"))

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-cudart", "static",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _stale(lib: str, deps) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in deps)


def _built_against() -> str:
    """What the extension module's machine code depends on beside its sources:
    it is compiled against torch's C++ interfaces, which change with torch."""
    import torch
    return f"torch {torch.__version__} abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} python {sys.version.split()[0]}"


def _binding_stale() -> bool:
    if _stale(LIB_BINDING, DEPS_BINDING) or not os.path.exists(LIB_BINDING + ".built"):
        return True
    with open(LIB_BINDING + ".built") as f:
        return f.read() != _built_against()


def stale() -> bool:
    return (_stale(LIB, DEPS + [HEADER]) or _stale(LIB_W4A16, DEPS_W4A16)
            or _stale(LIB_NVFP4, DEPS_NVFP4) or _stale(LIB_W4G, DEPS_W4G)
            or _stale(LIB_KV4, DEPS_KV4) or _binding_stale())


def _build_one(src: str, lib: str, verbose: bool) -> None:
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, src, "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)


def _build_binding(verbose: bool) -> None:
    """The extension module: plain C++ against torch's headers and the two
    libraries beside it (found through its own folder at run time; torch's own
    libraries are loaded with torch)."""
    import torch
    from torch.utils import cpp_extension
    tmp = LIB_BINDING + f".tmp{os.getpid()}"
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{p}" for p in cpp_extension.include_paths()), f"-I{cuda}", f"-I{sysconfig.get_paths()['include']}",
           SRC_BINDING, "-o", tmp, f"-L{torch_lib}", "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10",
           f"-L{HERE}", "-lconvrot_w4g", "-lconvrot_kv4", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_BINDING)
    with open(tmp, "w") as f:
        f.write(_built_against())
    os.replace(tmp, LIB_BINDING + ".built")


def build(force: bool = False, verbose: bool = False) -> str:
    """Build whichever library is missing or older than its sources, and the
    extension module also where it was built against another torch or Python;
    returns the W4A4 library's path."""
    if force or _stale(LIB, DEPS + [HEADER]):
        _build_one(SRC, LIB, verbose)
    if force or _stale(LIB_W4A16, DEPS_W4A16):
        _build_one(SRC_W4A16, LIB_W4A16, verbose)
    if force or _stale(LIB_NVFP4, DEPS_NVFP4):
        _build_one(SRC_NVFP4, LIB_NVFP4, verbose)
    if force or _stale(LIB_W4G, DEPS_W4G):
        _build_one(SRC_W4G, LIB_W4G, verbose)
    if force or _stale(LIB_KV4, DEPS_KV4):
        _build_one(SRC_KV4, LIB_KV4, verbose)
    if force or _binding_stale():
        _build_binding(verbose)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
    print(LIB_W4A16)
    print(LIB_NVFP4)
    print(LIB_W4G)
    print(LIB_KV4)
    print(LIB_BINDING)
