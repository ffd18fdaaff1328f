"""Build the CUDA library liblf_attn.so (nvcc, sm_100a) and the Python entry
of its paged-cache calls, _lf_bind.so (g++), in-tree.

    python -m sparse_sliding_window_b200.build
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "liblf_attn.so")
SOURCES = ["lf_api.cu", "lf_simt.cu", "lf_tc.cu", "lf_tc_bwd.cu", "lf_static.cu", "lf_gemm.cu",
           "lf_rope.cu", "lf_paged.cu", "lf_prefix.cu", "lf_prefix_tc.cu", "lf_paged_api.cu"]
BIND = os.path.join(HERE, "_lf_bind.so")
BIND_SOURCE = os.path.join(CSRC, "lf_bind.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-shared", "-Xptxas", "-warn-spills"]


def sources():
    return [os.path.join(CSRC, s) for s in SOURCES]


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    deps += [os.path.join(ROOT, "include", h) for h in ("lf_attn.h", "lf_proj.h", "lf_paged.h")]
    return any(os.path.getmtime(s) > t for s in deps)


def _bind_tag() -> bytes:
    """What the module carries of the torch that it was built against."""
    import torch
    return ("lf_bind for torch %s." % torch.__version__).encode()


def build_bind(force: bool = False, verbose: bool = False) -> str:
    """The Python module _lf_bind, against the installed torch and liblf_attn.so."""
    deps = [BIND_SOURCE] + [os.path.join(ROOT, "include", h) for h in ("lf_attn.h", "lf_paged.h")]
    tag = _bind_tag()
    if not force and os.path.exists(BIND) and all(os.path.getmtime(d) <= os.path.getmtime(BIND) for d in deps):
        with open(BIND, "rb") as f:
            if tag in f.read():
                return BIND
    from torch.utils import cpp_extension as ext
    tmp = BIND + ".tmp%d" % os.getpid()
    inc = ext.include_paths("cuda") + [sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    libs = ext.library_paths("cuda")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", '-DLF_BIND_TAG="%s"' % tag.decode(), "-o", tmp, BIND_SOURCE]
    for d in inc:
        cmd += ["-isystem" if d != inc[-1] else "-I", d]
    for d in libs:
        cmd += ["-L", d]
    cmd += ["-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L", HERE, "-l:liblf_attn.so",
            "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, BIND)
    return BIND


def build(force: bool = False, verbose: bool = False) -> str:
    """The library and, where torch and g++ are there for it, the Python entry
    of the paged-cache calls (build_bind raises where they are not)."""
    lib = build_lib(force, verbose)
    try:
        build_bind(force, verbose)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        warnings.warn("_lf_bind.so, the Python entry of the paged-cache calls, is not built: %r" % e)
    return lib


def build_lib(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [NVCC, *FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-o", tmp, *sources()]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
