"""Build libdecodegemm.so in-tree with nvcc for sm_103a (no cmake, parallel TUs), and the Python
marshalling module _marshal.so with g++ against the installed torch.  The library does not depend
on the module: it is linked whether or not that compiles."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import platform
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libdecodegemm.so")
OBJ = os.path.join(HERE, "_build")
PYSRC = os.path.join(HERE, "pybind", "_marshal.cpp")
PYMOD = os.path.join(HERE, "_marshal.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def build_id() -> str:
    """Content hash of every source and header, plus the compiler version."""
    h = hashlib.sha256()
    for f in sorted(glob.glob(os.path.join(CSRC, "*")) + [os.path.join(INCLUDE, "dg.h")]):
        with open(f, "rb") as fh:
            h.update(os.path.basename(f).encode() + b"\0" + fh.read())
    try:
        h.update(subprocess.run([_nvcc(), "--version"], capture_output=True, text=True).stdout.encode())
    except OSError:
        pass
    return h.hexdigest()[:16]


def _compile(src: str, bid: str) -> str:
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    cmd = [_nvcc(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
           f"-DDG_BUILD_ID=\"{bid}\"", "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _fresh(out: str, inputs) -> bool:
    return os.path.exists(out) and os.path.getmtime(out) >= max(os.path.getmtime(f) for f in inputs)


def _marshal_host() -> str:
    """What the Python module's ABI depends on; kept beside the module it was built for."""
    import torch
    return f"torch {torch.__version__}, Python {sys.version}, {platform.machine()}\n"


def _marshal_stamp() -> str:
    return os.path.join(OBJ, "_marshal.host")


def _marshal_fresh(inputs) -> bool:
    if not _fresh(PYMOD, inputs) or not os.path.exists(_marshal_stamp()):
        return False
    with open(_marshal_stamp()) as f:
        return f.read() == _marshal_host()


def _build_marshal() -> None:
    import torch
    from torch.utils import cpp_extension as ce
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [p for d in (*ce.include_paths(), os.path.join(home, "include"), sysconfig.get_path("include"), INCLUDE)
           for p in ("-I", d)]
    tmp = PYMOD + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *inc, PYSRC, "-o", tmp, f"-L{torch_lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           f"-Wl,-rpath,{torch_lib}", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {PYSRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, PYMOD)
    with open(_marshal_stamp(), "w") as f:
        f.write(_marshal_host())


def _build_lib(jobs: int | None) -> None:
    srcs = sources()
    bid = build_id()
    with cf.ThreadPoolExecutor(jobs or min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(lambda s: _compile(s, bid), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([_nvcc(), *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, jobs: int | None = None) -> str:
    header = os.path.join(INCLUDE, "dg.h")
    os.makedirs(OBJ, exist_ok=True)
    with cf.ThreadPoolExecutor(1) as ex:
        marshal = ex.submit(lambda: None if not force and _marshal_fresh([PYSRC, header]) else _build_marshal())
        if force or not _fresh(LIB, glob.glob(os.path.join(CSRC, "*")) + [header]):
            _build_lib(jobs)
        marshal.result()                   # (after the library is in place)
    return LIB


if __name__ == "__main__":
    print(build(force=True))
