"""Build libbcq.so (the sm_100a kernels behind the C ABI of include/bcq.h)
in-tree, next to this file, with nvcc.

Each translation unit of csrc/ is compiled to an object under _build/ (in
parallel; an object is rebuilt only when its source or a header it includes
changed), then the objects are linked.  The CUDA runtime is linked
statically and its symbols are kept private to the library, so the
process's other CUDA users (torch) are not affected.  Then the binding's fast
calls (csrc/bcq_fast.cpp, a CPython module over torch's headers) become
_fast.so next to it, with g++, where torch, its headers, Python's and the
compiler are there; the library and the binding work without.
"""
from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(ROOT, "_build", "libbcq")
LIB = os.path.join(HERE, "libbcq.so")
FAST_SRC = os.path.join(CSRC, "bcq_fast.cpp")
FAST = os.path.join(HERE, "_fast.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
          "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall"]
LFLAGS = ["-Xlinker", "--exclude-libs,ALL", "-Xlinker", "-Bsymbolic"]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _includes(path: str, seen: set) -> set:
    """Local headers (csrc/, include/) that `path` includes, transitively."""
    try:
        text = open(path).read()
    except OSError:
        return seen
    for name in re.findall(r'#include\s+"([^"]+)"', text):
        for d in (CSRC, INCLUDE):
            h = os.path.join(d, name)
            if os.path.exists(h) and h not in seen:
                seen.add(h)
                _includes(h, seen)
                break
    return seen


def _obj_of(src: str) -> str:
    return os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(nvcc: str, src: str, verbose: bool) -> str:
    obj = _obj_of(src)
    tmp = obj + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, *CFLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, obj)
    return obj


def build_fast(force: bool = False) -> str | None:
    """_fast.so against the torch of this interpreter (its headers and
    libraries' names; nothing of it is loaded).  None, and no module of an
    older build, where something that it takes is missing."""
    import importlib.util
    import sysconfig
    spec = importlib.util.find_spec("torch")
    torch_dir = os.path.dirname(spec.origin) if spec and spec.origin else ""
    python_h = os.path.join(sysconfig.get_paths()["include"], "Python.h")
    cxx = os.environ.get("CXX", "g++")
    for what, there in (("torch", torch_dir), ("torch's headers", os.path.isdir(os.path.join(torch_dir, "include"))),
                        (python_h, os.path.exists(python_h)), (cxx, shutil.which(cxx.split()[0]))):
        if not there:
            print(f"{os.path.basename(FAST)} is left out: no {what}", file=sys.stderr)
            if os.path.exists(FAST):
                os.unlink(FAST)
            return None
    version = os.path.join(torch_dir, "version.py")
    if force or _stale(FAST, [FAST_SRC, os.path.join(INCLUDE, "bcq.h"), version]):
        cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
        inc = [os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), os.path.dirname(python_h), INCLUDE]
        tmp = FAST + f".tmp{os.getpid()}"
        subprocess.run([*cxx.split(), "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
                        *[f"-I{d}" for d in inc], FAST_SRC, "-o", tmp,
                        "-L" + os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
                        "-ltorch_cuda", "-ltorch_python"], check=True)
        os.replace(tmp, FAST)
    return FAST


def build(force: bool = False, verbose: bool = False) -> str:
    nvcc = os.environ.get("NVCC", "nvcc")
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    todo = [s for s in srcs if force or _stale(_obj_of(s), [s, *_includes(s, set())])]
    if todo:
        with ThreadPoolExecutor(max_workers=len(todo)) as ex:
            list(ex.map(lambda s: _compile(nvcc, s, verbose), todo))
    objs = [_obj_of(s) for s in srcs]
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.run([nvcc, *ARCH, *LFLAGS, "-shared", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    build_fast(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
