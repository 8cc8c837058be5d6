"""Builds libnvfp4.so (the HIP kernels and the C ABI) in-tree for gfx950.

Every HIP source is compiled with hipcc for --offload-arch=gfx950 only; the
library is written next to this file so it travels with the source tree.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libnvfp4.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
# not part of the library: a test program and the bench's measurement probes,
# each built beside the file that uses it
CONFORMANCE_SRC = os.path.join(ROOT, "tests", "conformance_cvt.hip")
CONFORMANCE_PATH = os.path.join(ROOT, "tests", "conformance_cvt")
PROBES_SRC = os.path.join(ROOT, "bench_probes.hip")
PROBES_PATH = os.path.join(ROOT, "libnvfp4_probes.so")

SOURCES = ["nvfp4_abi.cpp", "quantize.hip", "fuse_rescale.hip", "gemm.hip", "gemm_fast.hip", "gemm_decode.hip", "gemm_stream.hip", "kv_quantize.hip",
           "nvfp4_kv_abi.cpp", "kv_table.hip", "rope.hip", "kv_cache_write.hip", "paged_attention.hip"]

# the native side of the paged KV cache's Python binding: an extension module
# beside the library, built against torch's headers (without torch: not at all,
# the C ABI does not need it)
BIND_SRC = "kv_bind.cpp"
BIND_PATH = os.path.join(HERE, "_kv_bind.so")

HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")

COMMON_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",  # the quantiser's fp32 steps are single IEEE operations, never fused
    "-fno-gpu-flush-denormals-to-zero",
    # packed fp32 VALU instructions are kept out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
    "-I", INCLUDE,
    "-I", CSRC,
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *COMMON_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return obj


def _compile_bind() -> str:
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths

    obj = os.path.join(BUILD_DIR, "kv_bind.o")
    includes = [INCLUDE, sysconfig.get_paths()["include"], *include_paths()]
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *(f"-I{p}" for p in includes), "-c", os.path.join(CSRC, BIND_SRC), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{CXX} failed for {BIND_SRC}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return obj


def _link_bind(obj: str):
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [CXX, "-shared", "-o", BIND_PATH + ".tmp", obj, "-L" + HERE, "-lnvfp4", "-Wl,-rpath,$ORIGIN", "-L" + libs,
           "-ltorch_python", "-ltorch_cpu", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(BIND_PATH + ".tmp", BIND_PATH)


def _has_torch() -> bool:
    try:
        import torch  # noqa: F401
    except ImportError:
        return False
    return True


def build(verbose: bool = False) -> str:
    """Compile every source and link libnvfp4.so, then the binding's module where torch is; returns the library path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as ex:
        bind = ex.submit(_compile_bind) if _has_torch() else None
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    # conformance check of the conversion instructions the kernels rely on
    # (a standalone program, run by the GPU tests)
    cmd = [HIPCC, *COMMON_FLAGS, CONFORMANCE_SRC, "-o", CONFORMANCE_PATH + ".tmp"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for conformance_cvt.hip:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(CONFORMANCE_PATH + ".tmp", CONFORMANCE_PATH)
    # measurement probes for the benchmark (MFMA-only loop, streaming read)
    cmd = [HIPCC, *COMMON_FLAGS, "-shared", PROBES_SRC, "-o", PROBES_PATH + ".tmp"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for bench_probes.hip:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(PROBES_PATH + ".tmp", PROBES_PATH)
    if verbose:
        print(f"built {LIB_PATH}, {CONFORMANCE_PATH} and {PROBES_PATH}")
    # last, so that nothing else is missing if it fails
    if bind is not None:
        _link_bind(bind.result())
    elif os.path.exists(BIND_PATH):
        os.remove(BIND_PATH)  # linked to an earlier library
    if verbose:
        print(f"built {BIND_PATH}" if bind is not None else f"no PyTorch: {BIND_PATH} is not built")
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True)
