"""Build liblqmm.so (HIP, gfx950) in-tree with hipcc, and the benchmark's
streaming-read probe (liblqmm_probe.so), and the native Python calls of the
serving operators (_serve.so, against torch's headers).

Each source is compiled to an object in parallel, then the objects are linked
into the shared library.

Usage: python -m block_quantized_matmul_amd.build
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "liblqmm.so")
SOURCES = ["api.hip", "gemv.hip", "gemv_small.hip", "gemv_small_more.hip", "gemm_q8_0.hip",
           "gemm_lds.hip", "sgemm.hip", "gemv_whole.hip", "api_serve.hip", "kv_append.hip",
           "attn_prefix.hip", "f8b128.hip", "kv_append_norm.hip", "kv_read_f8.hip", "attn_f8.hip",
           "mxfp4.hip"]
PROBE_LIB = os.path.join(HERE, "liblqmm_probe.so")
PROBE_SOURCES = ["probe.hip"]
BINDING = os.path.join(HERE, "_serve.so")
BINDING_SOURCE = "serve_binding.cpp"
CXX = os.environ.get("CXX", "g++")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # no packed-fp32 VALU instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-result",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def _run(cmd, what, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed building {what}")
    err = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l
                    and "not a recognized feature" not in l)
    if verbose and err.strip():
        sys.stderr.write(err + "\n")


def _hipcc(sources, lib, verbose):
    os.makedirs(OBJ, exist_ok=True)
    objs = [os.path.join(OBJ, os.path.splitext(s)[0] + ".o") for s in sources]
    jobs = [([HIPCC, *FLAGS, "-c", os.path.join(CSRC, s), "-o", o], s, verbose)
            for s, o in zip(sources, objs)]
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
        for f in [ex.submit(_run, *j) for j in jobs]:
            f.result()
    tmp = lib + ".tmp"
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp],
         os.path.basename(lib), verbose)
    os.replace(tmp, lib)
    return lib


def _binding(verbose):
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    tmp = BINDING + ".tmp"
    _run([CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"],
          "-isystem", os.path.join(root, "include"),
          "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
          os.path.join(CSRC, BINDING_SOURCE), "-o", tmp,
          "-L", HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
          "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10"],
         BINDING_SOURCE, verbose)
    os.replace(tmp, BINDING)


def build(verbose: bool = False) -> str:
    _hipcc(PROBE_SOURCES, PROBE_LIB, verbose)
    lib = _hipcc(SOURCES, LIB, verbose)
    _binding(verbose)
    return lib


if __name__ == "__main__":
    print(build(verbose=True))
