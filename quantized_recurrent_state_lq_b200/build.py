"""Build liblq.so (the CUDA library behind include/lq_state.h) in-tree.

nvcc compiles every csrc/*.cu for sm_100a only and links them, with the CUDA
runtime linked statically, into quantized_recurrent_state_lq_b200/liblq.so;
g++ compiles csrc/lq_bind.cpp (host code, against torch) into _bind.<Python>.<torch>.so
beside it.
Run `python -m quantized_recurrent_state_lq_b200.build` or call build() and
build_bind(); the binding is built where its calls are first made if it is
missing, the library alone needs no host compiler for torch's headers.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "liblq.so")
BIND_SRC = os.path.join(CSRC, "lq_bind.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-cudart", "static",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(OUT):
        return True
    t = os.path.getmtime(OUT)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    deps.append(os.path.join(ROOT, "include", "lq_state.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def bind_path() -> str:
    """The binding for this Python and this torch: both are named in the file,
    since one compiled against another's headers may load and misread tensors."""
    import sysconfig

    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(HERE, f"_bind.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}-abi{abi}.so")


def bind_stale() -> bool:
    out = bind_path()
    if not os.path.exists(out):
        return True
    deps = [BIND_SRC, os.path.join(ROOT, "include", "lq_state.h")]
    return any(os.path.getmtime(d) > os.path.getmtime(out) for d in deps)


def _bind_command(out: str) -> list[str]:
    import sysconfig

    import torch
    tdir = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(shutil.which(NVCC) or NVCC))
    inc = [os.path.join(tdir, "include"), os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + os.path.join(ROOT, "include"),
            "-I" + sysconfig.get_paths()["include"], *(a for d in inc for a in ("-isystem", d)), BIND_SRC,
            "-L" + os.path.join(tdir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-o", out]


def build_bind(verbose: bool = False) -> str:
    """Compiles into a file of this call's own, so that ranks that build at the
    same time each put a whole one in place."""
    out = bind_path()
    fd, tmp = tempfile.mkstemp(prefix="_bind.", suffix=".tmp.so", dir=HERE)
    os.close(fd)
    try:
        cmd = _bind_command(tmp)
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.chmod(tmp, 0o755)
        os.replace(tmp, out)
    except BaseException:
        os.unlink(tmp)
        raise
    return out


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and not _stale():
        return OUT
    objs = []
    bdir = os.path.join(HERE, "_build")
    os.makedirs(bdir, exist_ok=True)
    procs = []
    for src in sources():
        obj = os.path.join(bdir, os.path.basename(src) + ".o")
        cmd = [NVCC, *ARCH, *FLAGS, *(extra or []), "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((subprocess.Popen(cmd), cmd))
        objs.append(obj)
    for p, cmd in procs:
        if p.wait() != 0:
            raise RuntimeError("nvcc failed: " + " ".join(cmd))
    tmp = OUT + ".tmp"
    cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    subprocess.run(cmd, check=True)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None)
    if "--force" in sys.argv or bind_stale():
        build_bind(verbose=True)
    print(OUT)
