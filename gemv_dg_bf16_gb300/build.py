"""Build libdecodegemm.so in-tree with nvcc for sm_103a (no cmake, parallel TUs), and the Python
marshalling module _marshal.so with g++ against the installed torch."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import subprocess
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


def build(force: bool = False, jobs: int | None = None) -> str:
    srcs = sources()
    header = os.path.join(INCLUDE, "dg.h")
    lib_ok = not force and _fresh(LIB, glob.glob(os.path.join(CSRC, "*")) + [header])
    py_ok = not force and _fresh(PYMOD, [PYSRC, header])
    if lib_ok and py_ok:
        return LIB
    if lib_ok:
        _build_marshal()
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    bid = build_id()
    jobs = jobs or min(len(srcs), os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(jobs + 1) as ex:
        marshal = None if py_ok else ex.submit(_build_marshal)
        objs = list(ex.map(lambda s: _compile(s, bid), srcs))
        if marshal:
            marshal.result()
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([_nvcc(), *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True))
