"""Compile libzha.so (the C-ABI CUDA library) in-tree for sm_100a with nvcc, and _bind.so (argument marshalling of the
paged and rotary calls, over torch's C++ headers) with the host compiler."""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libzha.so")
BIND_SRC = os.path.join(CSRC, "zha_bind.cpp")
BIND = os.path.join(HERE, "_bind.so")
BIND_KEY = os.path.join(HERE, "_build", "_bind.key")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++20",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
         "-I", INCLUDE]


# Per-file flags. The tree kernels compute the same planes in several kernels
# (bulk build, appends, the decode step's rightmost path) and must agree bit
# for bit: no implicit a*b+c contraction there (every FMA is written out).
FILE_FLAGS = {"zha_tree.cu": ["--fmad=false"]}


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return (glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
            glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + headers()
    return any(os.path.getmtime(p) > t for p in deps)


def bind_key() -> str:
    """What _bind.so is built for: its tensors and objects are those of one torch and one Python."""
    import torch
    return "torch %s, C++11 ABI %d, Python %s" % (torch.__version__, int(torch._C._GLIBCXX_USE_CXX11_ABI),
                                                  sysconfig.get_config_var("EXT_SUFFIX"))


def _bind_stale() -> bool:
    if not os.path.exists(BIND) or not os.path.exists(BIND_KEY):
        return True
    with open(BIND_KEY) as f:
        if f.read() != bind_key():
            return True
    newest = max(os.path.getmtime(p) for p in [BIND_SRC] + glob.glob(os.path.join(INCLUDE, "*.h")))
    return os.path.getmtime(BIND) <= newest


def build_bind(force: bool = False, verbose: bool = False) -> str:
    if not force and not _bind_stale():
        return BIND
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    tmp = BIND + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           '-DZHA_BIND_KEY="%s"' % bind_key(), "-I", INCLUDE]
    for inc in (os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]):
        cmd += ["-isystem", inc]
    cmd += [BIND_SRC, "-o", tmp, "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
            "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, BIND)
    os.makedirs(os.path.dirname(BIND_KEY), exist_ok=True)
    with open(BIND_KEY, "w") as f:
        f.write(bind_key())
    return BIND


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    build_bind(force, verbose)
    if not force and not _stale():
        return LIB
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    newest_header = max((os.path.getmtime(h) for h in headers()), default=0.0)
    objs, cmds = [], []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        objs.append(obj)
        fresh = (os.path.exists(obj) and not force and not extra and
                 os.path.getmtime(obj) > max(os.path.getmtime(src), newest_header))
        if not fresh:
            cmds.append([NVCC, *FLAGS, *FILE_FLAGS.get(os.path.basename(src), []), *extra, "-c", src, "-o", obj])
    # the translation units are independent: compile them side by side
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(cmds), os.cpu_count() or 1))) as ex:
        for cmd in cmds:
            if verbose:
                print(" ".join(cmd), flush=True)
        for f in [ex.submit(subprocess.check_call, cmd) for cmd in cmds]:
            f.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    subprocess.check_call([NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp,
                           *objs, "-lcudart"])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
