"""Build the CUDA library ``libcoli_moe.so`` in-tree for sm_100a."""
from __future__ import annotations

import glob
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
SO = os.path.join(HERE, "libcoli_moe.so")
BINDING_SO = os.path.join(HERE, "_binding.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
    "-Xcompiler", "-fPIC,-fvisibility=hidden", "-shared", "--expt-relaxed-constexpr",
    "-Xlinker", "-soname=" + os.path.basename(SO),  # a name, not this machine's path, in what links to it
]


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    """COLI_TC_TRACE=1 in the environment builds the profiling variant whose
    tensor-core kernels record a block timeline into the trace buffer."""
    srcs = sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))
    flags = list(extra or [])
    if os.environ.get("COLI_TC_TRACE") == "1":
        flags.append("-DCOLI_TC_TRACE=1")
    cmd = ["nvcc", "-t", "0", *NVCC_FLAGS, *flags, "-o", SO, *srcs]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    build_binding(verbose)
    return SO


def build_binding(verbose: bool = False) -> str | None:
    """The Python module of the operators on torch tensors (csrc/binding.cpp), linked by name to the libcoli_moe.so
    beside it: a copied or moved package runs its own library. Only these operators need it: without torch, its CUDA
    libraries or Python's headers it is left out (None), and the C library and its ctypes layer are all there is."""
    import importlib.util
    import sysconfig

    spec = importlib.util.find_spec("torch")
    missing = None
    if spec is None or not spec.origin:
        missing = "torch is not installed"
    elif not glob.glob(os.path.join(os.path.dirname(spec.origin), "lib", "libc10_cuda.so*")):
        missing = "torch was built without CUDA"
    elif not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        missing = "Python.h is not installed"
    if missing:
        print(f"{os.path.basename(BINDING_SO)} is not built: {missing}; the operators on torch tensors are not available")
        return None
    torch = os.path.dirname(spec.origin)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(torch, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           *(x for i in inc for x in ("-isystem", i)),
           os.path.join(HERE, "csrc", "binding.cpp"), "-o", BINDING_SO, "-L" + HERE, "-l:" + os.path.basename(SO), "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch",
           "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    return BINDING_SO


if __name__ == "__main__":
    build(verbose=True)
