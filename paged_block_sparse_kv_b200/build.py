"""Build libvx.so (the C-ABI CUDA library) in-tree with nvcc for sm_100a, and _vx_marshal (argument marshalling of
the 8-bit cache and page calls for Python, C++ against torch's headers) beside it.

    python -m paged_block_sparse_kv_b200.build [--force] [--verbose]

The CUDA runtime is linked statically so the library does not depend on which
libcudart another component of the process (e.g. torch) brought in; the driver API
entry point for TMA descriptors is fetched through the runtime at first use.
"""
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libvx.so")
MARSHAL = os.path.join(HERE, "_vx_marshal.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-O2",
         "-I" + os.path.join(ROOT, "include")]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def marshal_mark() -> str:
    """What _vx_marshal.so was built for: its docstring.  Its layout of tensors is that of one torch, one Python."""
    import torch
    return f"vx marshal for torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"


def _marshal_stale():
    if not os.path.exists(MARSHAL):
        return True
    t = os.path.getmtime(MARSHAL)
    if any(os.path.getmtime(p) > t for p in (MARSHAL_SRC, os.path.join(ROOT, "include", "vx.h"))):
        return True
    with open(MARSHAL, "rb") as f:
        return marshal_mark().encode() + b"\0" not in f.read()


def build_marshal(force: bool = False) -> str:
    if not force and not _marshal_stale():
        return MARSHAL
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    tmp = MARSHAL + ".tmp"
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-o", tmp, MARSHAL_SRC,
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                    f'-DVX_MARSHAL_MARK="{marshal_mark()}"',
                    "-I" + sysconfig.get_paths()["include"], "-isystem", os.path.join(base, "include"),
                    "-isystem", os.path.join(cuda, "include"), "-L" + os.path.join(base, "lib"),
                    "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"], check=True)
    os.replace(tmp, MARSHAL)
    return MARSHAL


def build(force: bool = False, verbose: bool = False) -> str:
    build_marshal(force)
    if not force and not _stale():
        return LIB
    objdir = os.path.join(ROOT, "_build", "libvx")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    subprocess.run([NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
