"""Build the CUDA library (libspecverify.so) in-tree for sm_103a with nvcc.

Each translation unit compiles in its own nvcc process (in parallel), then the
objects link into one shared library next to this file.  No CMake, no torch
extension machinery: the library exports a plain C ABI (include/spec_verify.h).
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libspecverify.so")
CALLS = os.path.join(PKG, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]

SOURCES = ["api.cu", "kv_cache.cu", "verify.cu", "verify_bf16.cu", "verify_f32.cu", "verify_mixed.cu",
           "verify_static.cu", "verify_topk_bf16.cu", "verify_topk_f32.cu", "verify_topk_mixed.cu",
           "tree_verify.cu", "tree_bf16.cu", "tree_f32.cu", "tree_opts_bf16.cu", "tree_opts_f32.cu",
           "stream.cu", "stream_more.cu", "tree_mask.cu", "kv_entries.cu", "logit_rules.cu",
           "tree_attention.cu", "attention_bf16.cu", "attention_e4m3.cu"]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _build_calls() -> None:
    """The Python side of the per-layer calls (csrc/calls.cpp): a plain
    extension module over torch's tensor type."""
    import sysconfig

    import torch
    root = os.path.join(os.path.dirname(torch.__file__))
    inc = os.path.join(root, "include")
    cmd = [shutil.which("g++") or "g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + INCLUDE, "-I" + inc,
           "-I" + os.path.join(inc, "torch", "csrc", "api", "include"), "-I" + sysconfig.get_paths()["include"],
           os.path.join(CSRC, "calls.cpp"), "-o", CALLS + ".tmp", "-L" + os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-ldl", "-Wl,-rpath," + os.path.join(root, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(CALLS + ".tmp", CALLS)


def build(verbose: bool = False, extra=(), out: str = LIB, only=None) -> str:
    """Compile the sources and link `out` (default: the package's library).
    `extra` nvcc flags apply to the translation units compiled; with `only`,
    just those sources are recompiled and the others' objects are reused."""
    os.makedirs(BUILD, exist_ok=True)
    todo = SOURCES if only is None else [s for s in SOURCES if s in only]
    with cf.ThreadPoolExecutor(max_workers=len(todo) + 1) as ex:
        calls = ex.submit(_build_calls) if only is None else None
        list(ex.map(lambda s: _compile(s, list(extra)), todo))
    objs = [os.path.join(BUILD, os.path.splitext(s)[0] + ".o") for s in SOURCES]
    tmp = out + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    if calls is not None:
        calls.result()  # the library stands without it
    if verbose:
        print("built", out, file=sys.stderr)
    return out


if __name__ == "__main__":
    build(verbose=True)
