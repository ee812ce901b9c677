"""Build librtp.so (the CUDA library behind include/rtp.h and rtp_paged.h) in-tree for sm_100a, and,
where torch is installed, _paged.so, the torch binding of the paged-cache operators."""
import glob
import importlib.metadata
import importlib.util
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "librtp.so")
EXT = os.path.join(PKG, "_paged.so")
EXT_FOR = os.path.join(PKG, "_paged.torch")  # what the binding was built for: it uses torch's internals
EXT_SOURCE = os.path.join(CSRC, "paged_torch.cpp")
CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2", "-shared", "-cudart", "static",
    "--expt-relaxed-constexpr",
    "-I", INCLUDE, "-I", CSRC,
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    deps += glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _torch() -> str:
    """The torch and the interpreter that a binding is for; empty without torch."""
    if importlib.util.find_spec("torch") is None:
        return ""
    return f"torch {importlib.metadata.version('torch')} {sys.implementation.cache_tag}\n"


def build_binding(force: bool = False):
    """The torch binding: links to librtp.so beside it and to torch.  None without torch: the C
    library does without it."""
    built_for = _torch()
    if not built_for:
        print("torch is not installed: PagedKV's binding is not built", file=sys.stderr)
        return None
    deps = [EXT_SOURCE] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if (not force and os.path.exists(EXT) and os.path.exists(EXT_FOR) and open(EXT_FOR).read() == built_for
            and all(os.path.getmtime(d) <= os.path.getmtime(EXT) for d in deps)):
        return EXT
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ce

    cmd = [CXX, "-shared", "-fPIC", "-O2", "-std=c++17", "-w", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-DTORCH_EXTENSION_NAME=_paged", "-I", INCLUDE, "-isystem", sysconfig.get_paths()["include"]]
    for d in ce.include_paths("cuda"):
        cmd += ["-isystem", d]
    cmd += ["-o", EXT, EXT_SOURCE, "-L", PKG, "-l:librtp.so", "-Wl,-rpath,$ORIGIN"]
    for d in ce.library_paths("cuda"):
        cmd += ["-L", d]
    cmd += ["-lc10", "-lc10_cuda", "-lcudart", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    subprocess.check_call(cmd)
    with open(EXT_FOR, "w") as f:
        f.write(built_for)
    return EXT


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        build_binding()
        return LIB
    cmd = [NVCC] + FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-o", LIB] + sources()
    subprocess.check_call(cmd)
    build_binding(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
