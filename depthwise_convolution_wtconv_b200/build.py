"""Builds libwtconv.so in-tree for sm_100a with nvcc.

    python -m depthwise_convolution_wtconv_b200.build
"""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")          # the image layer
CSRC_SEQ = os.path.join(PKG, "csrc_seq")  # the sequence operators
SRC = [os.path.join(CSRC, "wtconv_api.cu"), os.path.join(CSRC_SEQ, "seq_api.cu")]
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libwtconv.so")


def _files(*dirs):
    return [os.path.join(d, f) for d in dirs for f in os.listdir(d)]


def _deps(src):
    headers = ["wtconv.h"] + (["wtconv_seq.h"] if os.path.dirname(src) == CSRC_SEQ else [])
    return _files(os.path.dirname(src)) + [os.path.join(INCLUDE, h) for h in headers]


def _object(src):
    return os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")


def nvcc_command(src, verbose=False):
    cmd = [
        "nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
        "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + os.path.dirname(src), "-c", src, "-o", _object(src),
    ]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    return cmd


def _newer(target, deps):
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in deps)


def up_to_date():
    return _newer(LIB, [p for s in SRC for p in _deps(s)])


def build(force=False, verbose=False):
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    stale = [s for s in SRC if force or not _newer(_object(s), _deps(s))]
    with ThreadPoolExecutor(len(SRC)) as pool:
        list(pool.map(lambda s: subprocess.run(nvcc_command(s, verbose), check=True), stale))
    subprocess.run(["nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", LIB] +
                   [_object(s) for s in SRC], check=True)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
