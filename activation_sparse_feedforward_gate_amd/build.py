"""Build libtwell.so in-tree: every HIP/C++ source under csrc/ is compiled for
gfx950 with hipcc and linked into activation_sparse_feedforward_gate_amd/lib/;
and after it _twell_bind, the Python module that marshals tensors for some of
its calls (csrc/bind.cpp, host code), where torch and its headers are there: the
library itself and its C ABI need hipcc alone.

    python -m activation_sparse_feedforward_gate_amd.build [--jobs N]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libtwell.so")
BIND = os.path.join(LIBDIR, "_twell_bind.so")
ROOT = os.path.dirname(PKG)

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
# Packed fp32 VALU ops are switched off for every HIP translation unit.
CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"), "-Wall", "-Wno-unused-function",
]
SOURCES = ["twell_api.cpp", "twell_gate.hip", "twell_sparse.hip", "twell_sparse_bf16.hip", "twell_union.hip", "twell_hybrid.hip", "dense_ffn.hip", "dense_train.hip", "twell_decode.hip", "twell_compact.hip",
           "block_api.cpp", "block_norm.hip", "block_w4.hip"]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CFLAGS, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stderr}")
    return obj


def _build_bind() -> None:
    import torch
    from torch.utils.cpp_extension import include_paths
    obj, tmp = os.path.join(BUILD, "bind.o"), BIND + ".tmp"
    inc = [*include_paths(), sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "include"),
           os.path.join(ROOT, "include")]
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    for what, cmd in (
            ("compile", [HIPCC, "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
                         "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
                         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                         *[f for i in inc for f in ("-isystem", i)], "-c", os.path.join(CSRC, "bind.cpp"), "-o", obj]),
            ("link", [HIPCC, "-shared", "-no-hip-rt", "-o", tmp, obj, "-L" + LIBDIR, "-ltwell", "-L" + tlib, "-ltorch_python", "-ltorch",
                      "-ltorch_cpu", "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN"])):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} of bind.cpp failed:\n{r.stderr}")
    os.replace(tmp, BIND)


def build(jobs: int = 8, verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=max(1, jobs)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    try:
        import torch  # noqa: F401
    except ImportError:
        print("torch is not importable: the Python module that marshals its tensors is not built")
        return LIB
    _build_bind()
    if verbose:
        print(f"built {BIND}")
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=min(8, os.cpu_count() or 1))
    args = ap.parse_args(argv)
    build(args.jobs)
    return 0


if __name__ == "__main__":
    sys.exit(main())
