"""Builds libqkvfront.so in-tree with nvcc for sm_103a (no other arch)."""
from __future__ import annotations

import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = [os.path.join(PKG, "csrc", "qkv_front.cu")]
HEADERS = [os.path.join(ROOT, "include", "qkvfront.h"),
           os.path.join(PKG, "csrc", "qknorm_rope_kv_insert.cuh"),
           os.path.join(PKG, "csrc", "layer_front.cuh"),
           os.path.join(PKG, "csrc", "attn2.cuh"),
           os.path.join(PKG, "csrc", "rope.cuh"),
           os.path.join(PKG, "csrc", "rope_kv_append.cuh"),
           os.path.join(PKG, "csrc", "prefix_plan.h"),
           os.path.join(PKG, "csrc", "prefix_attn.cuh")]
LIB_PATH = os.path.join(PKG, "libqkvfront.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
]


def nvcc_path() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libqkvfront")
    return cand


def stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    built = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(f) > built for f in SOURCES + HEADERS + [__file__])


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if missing or older than its sources; returns its path."""
    if not force and not stale():
        return LIB_PATH
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc_path(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-o", tmp, *SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH
