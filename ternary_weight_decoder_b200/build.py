"""Build ``libternary_decoder.so`` (sm_100a) in-tree with nvcc.

Each ``csrc/*.cu`` is compiled to ``_build/*.o`` (rebuilt when it or any
header under ``csrc/`` or ``include/`` is newer), then linked with the static
CUDA runtime into ``libternary_decoder.so`` next to this file.
``csrc/tw_bind.cpp``, the argument marshalling that works on torch tensors,
becomes the extension module ``_bind.so`` beside it (the host compiler and
torch's own headers and libraries; rebuilt for another torch or Python too).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libternary_decoder.so")
BIND = os.path.join(PKG, "_bind.so")
BIND_MADE_FOR = os.path.join(BUILD, "bind.made_for")   # the torch, Python and CUDA of that

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden",
                     "-I", os.path.join(ROOT, "include")]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _newest(paths):
    return max((os.path.getmtime(p) for p in paths), default=0.0)


def bind_made_for() -> str:
    """What the extension module's binary interface depends on beside its source."""
    return "\n".join(["torch " + importlib.metadata.version("torch"), str(sysconfig.get_config_var("SOABI")),
                      _nvcc()])


def bind_is_current() -> bool:
    if not os.path.exists(BIND) or not os.path.exists(BIND_MADE_FOR):
        return False
    with open(BIND_MADE_FOR) as f:
        if f.read() != bind_made_for():
            return False
    return os.path.getmtime(BIND) >= _newest([os.path.join(CSRC, "tw_bind.cpp")] +
                                             glob.glob(os.path.join(ROOT, "include", "*.h")))


def build_bind() -> None:
    if bind_is_current():
        return
    src = os.path.join(CSRC, "tw_bind.cpp")
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(base, "include"),
           "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(cuda or "/usr/local/cuda", "include"), src, "-o", tmp,
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
           "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("g++ failed: " + " ".join(cmd))
    os.replace(tmp, BIND)
    with open(BIND_MADE_FOR, "w") as f:
        f.write(bind_made_for())


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    hdr_time = _newest(headers)
    nvcc = _nvcc()
    jobs = []
    objs = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if ptxas_info or not os.path.exists(obj) or \
                os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_time):
            cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", obj]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
            for cmd, r in ex.map(run, jobs):
                if verbose or ptxas_info or r.returncode:
                    sys.stderr.write(r.stdout + r.stderr)
                if r.returncode:
                    raise RuntimeError("nvcc failed: " + " ".join(cmd))
    if jobs or not os.path.exists(LIB) or os.path.getmtime(LIB) < _newest(objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(tmp, LIB)
    build_bind()   # last: without it the library serves all but the cache operators and the norms
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="-v" in sys.argv))
