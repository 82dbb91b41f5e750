"""Builds librtp.so in-tree: host C++ with g++, CUDA with nvcc for sm_103a only.

Translation units compile in parallel; the result links the CUDA runtime
statically. A small Python extension (_table.so) is built beside it. Object files go to ``_build/`` next to this file.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "librtp.so")
TABLE = os.path.join(HERE, "_table.so")  # Python extension: pointer tables of checked tensors

HOST_SOURCES = ["spec.cpp", "plan.cpp", "infer.cpp"]
CUDA_SOURCES = ["boxing.cu", "tp_mlp.cu", "tp_mlp_static.cu", "linear.cu", "linear_gemm.cu", "linear_gemm_split.cu", "linear_few.cu", "grad_norm.cu", "cross_entropy.cu",
                "adamw.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _deps() -> list:
    files = [os.path.join(INCLUDE, "rtp.h")]
    for f in os.listdir(CSRC):
        files.append(os.path.join(CSRC, f))
    return files


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _table_command(target: str) -> list:
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext

    inc = [a for p in ext.include_paths() + [sysconfig.get_paths()["include"]] for a in ("-isystem", p)]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-shared", *inc, "-I", INCLUDE,
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, os.path.join(CSRC, "table.cpp"), "-o", target,
            "-L", ext.library_paths()[0], "-lc10", "-ltorch_cpu", "-ltorch_python"]


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    deps = _deps() + [os.path.abspath(__file__)]
    if not force and not _stale(LIB, deps) and not _stale(TABLE, deps):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    procs, objs = [], []
    for src in HOST_SOURCES:
        obj = os.path.join(BUILD, src + ".o")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    for src in CUDA_SOURCES:
        obj = os.path.join(BUILD, src + ".o")
        cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
               "-c", os.path.join(CSRC, src), "-o", obj]
        if ptxas_info:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    table_tmp, tmp = (f + ".tmp%d" % os.getpid() for f in (TABLE, LIB))
    try:
        cmd = _table_command(table_tmp)
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        failed = []
        for cmd, p in procs:
            out, _ = p.communicate()
            text = out.decode(errors="replace")
            if p.returncode != 0:
                failed.append((cmd, text))
            elif verbose and text.strip():
                sys.stderr.write(text)
        if failed:
            msg = "\n".join(" ".join(c) + "\n" + t for c, t in failed)
            raise RuntimeError("librtp build failed:\n" + msg)
        subprocess.check_call([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
        os.replace(table_tmp, TABLE)
    finally:  # a build that failed or was interrupted leaves neither compilers nor files behind
        for _, p in procs:
            if p.poll() is None:
                p.kill()
            p.wait()
        for f in (table_tmp, tmp):
            if os.path.exists(f):
                os.remove(f)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="-v" in sys.argv))
