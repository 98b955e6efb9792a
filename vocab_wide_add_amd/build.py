"""Build the gfx950 C-ABI library ``libxpress_argmax.so`` in-tree with hipcc, and
beside it ``_marshal.so``, the host code that fills the serving operators' argument
structs from torch tensors.

Usage: ``python -m vocab_wide_add_amd.build`` (or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRCS = [os.path.join(PKG, "csrc", "xpress_argmax.hip"),
        os.path.join(PKG, "csrc", "readout_gemm.hip"),
        os.path.join(PKG, "csrc", "latent.hip"),
        os.path.join(PKG, "csrc", "kv_append.hip"),
        os.path.join(PKG, "csrc", "paged_attention.hip"),
        os.path.join(PKG, "csrc", "sparse_attention.hip"),
        os.path.join(PKG, "csrc", "wide_attention.hip"),
        os.path.join(PKG, "csrc", "kv_pages.hip"),
        os.path.join(PKG, "csrc", "beams.hip"),
        os.path.join(PKG, "csrc", "sample.hip"),
        os.path.join(PKG, "csrc", "read_probe.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libxpress_argmax.so")
MARSHAL_SRC = os.path.join(PKG, "csrc", "marshal.cpp")
MARSHAL = os.path.join(PKG, "_marshal.so")
JOBS = max(1, min(8, os.cpu_count() or 1))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # IEEE behaviour the readout depends on: no flush of fp32 denormals, no
    # fast-math reassociation.
    "-fno-gpu-flush-denormals-to-zero",
    "-fno-fast-math",
    # packed fp32 VALU ops stay off (plain v_add_f32 / v_cvt_pk_bf16_f32 only)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


def _run(cmd, out: str, verbose: bool) -> None:
    """Compile to a file beside `out`, then put it in place."""
    tmp = out + ".tmp%d" % os.getpid()
    cmd = [tmp if x == out else x for x in cmd]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)


def build_marshal(verbose: bool = False) -> str:
    """Compile the host module against torch's headers (always recompiles)."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
          "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-I", INCLUDE,
          "-isystem", sysconfig.get_paths()["include"], "-isystem", "/opt/rocm/include"]
         + [x for d in include_paths() for x in ("-isystem", d)]
         + ["-o", MARSHAL, MARSHAL_SRC, "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"],
         MARSHAL, verbose)
    return MARSHAL


def build(verbose: bool = False) -> str:
    """Compile the library and the host module; returns the library's path
    (always recompiles).  The sources are compiled side by side: the three forms of
    the attention take one to two and a half minutes each."""
    with tempfile.TemporaryDirectory(dir=PKG, prefix="build_") as tmp, \
            concurrent.futures.ThreadPoolExecutor(JOBS) as pool:
        objects = [os.path.join(tmp, os.path.basename(src) + ".o") for src in SRCS]
        jobs = [pool.submit(build_marshal, verbose)]
        jobs += [pool.submit(_run, [HIPCC] + FLAGS + ["-I", INCLUDE, "-c", "-o", obj, src], obj, verbose)
                 for src, obj in zip(SRCS, objects)]
        for job in jobs:
            job.result()
        _run([HIPCC] + FLAGS + ["-shared", "-o", LIB] + objects, LIB, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
    sys.exit(0)
