"""Build libgdn.so (the C-ABI library) in-tree with hipcc for gfx950, and _bind.so (host code only: the argument
marshalling of the softmax-attention operators) against torch's headers.

Every source of libgdn.so under csrc/ is compiled to an object in _build/ (in parallel), then linked into
gated_delta_rule_varlen_amd/libgdn.so.  Run as ``python -m gated_delta_rule_varlen_amd.build``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdn.so")
BIND = os.path.join(PKG, "_bind.so")
SOURCES = ["gdn_api.cpp", "gdn_conv.hip", "gdn_prepare.hip", "gdn_scan.hip", "gdn_seq.hip", "gdn_chunk.hip",
           "gdn_chunk_k64.hip", "gdn_chunk_k128.hip", "gdn_chunk_k256.hip",
           "gdn_decode.hip", "gdn_noalloc.hip", "gdn_attn_api.cpp", "gdn_rope.hip", "gdn_attn.hip",
           "gdn_attn_bf16.hip", "gdn_attn_f16.hip", "gdn_attn_f32.hip"]

HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # packed fp32 VALU forms are kept out of generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
    "-I", CSRC,
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _build_bind() -> None:
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    tmp = BIND + f".tmp{os.getpid()}"
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(HIPCC)))
    dirs = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], os.path.join(ROOT, "include"),
                                            os.path.join(rocm, "include"), "/opt/rocm/include"]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
           "-D__HIP_PLATFORM_AMD__=1", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(x for d in dirs for x in ("-isystem", d)), os.path.join(CSRC, "gdn_bind.cpp"), "-o", tmp, "-L" + libs,
           "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for gdn_bind.cpp:\n{r.stderr}")
    os.replace(tmp, BIND)


def build(verbose: bool = False) -> str:
    """Compile every HIP source and link libgdn.so, and the binding beside it; returns the library path.  Where the
    binding does not compile libgdn.so is linked all the same, and then the error is raised."""
    os.makedirs(BUILD, exist_ok=True)
    jobs = min(len(SOURCES), int(os.environ.get("MAX_JOBS", os.cpu_count() or 4)))
    with ThreadPoolExecutor(max_workers=max(1, jobs)) as ex:
        bind = ex.submit(_build_bind)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}", flush=True)
    bind.result()  # only now: the library needs neither a host compiler nor torch's headers
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
