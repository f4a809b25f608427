"""Build libkd.so in-tree for sm_100a with nvcc, and, where torch is installed, _kd_torch.so, the operators on
torch tensors, with g++ against it and the installed torch (no JIT cache)."""

import importlib.metadata
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libkd.so")
TORCH_OUT = os.path.join(HERE, "_kd_torch.so")
TORCH_STAMP = os.path.join(ROOT, "_build", "torch_version")  # the torch that _kd_torch.so was built with
TORCH_SOURCE = os.path.join(CSRC, "kd_torch.cpp")
SOURCES = ["kd_kernel.cu", "kd_api.cu", "kd_noalloc.cu", "kd_gemm.cu", "kd_attention.cu",
           "kd_prefill.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _build_lib(force, verbose):
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")]
    deps += [os.path.join(ROOT, "include", "kd.h"), os.path.abspath(__file__)]
    if not force and not _stale(OUT, deps):
        return
    bdir = os.path.join(ROOT, "_build")
    os.makedirs(bdir, exist_ok=True)
    jobs = []
    for src in SOURCES:
        obj = os.path.join(bdir, src.replace(".cu", ".o"))
        cmd = [NVCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        jobs.append((obj, cmd, subprocess.Popen(cmd)))
    failed = [cmd for _, cmd, p in jobs if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    tmp = OUT + ".tmp%d" % os.getpid()
    subprocess.check_call([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp,
                           *[obj for obj, _, _ in jobs]])
    os.replace(tmp, OUT)


def _torch_version():
    """Of the installed torch, without importing it; None without one."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None


def _torch_stale(version):
    deps = [TORCH_SOURCE, os.path.join(ROOT, "include", "kd.h"), os.path.abspath(__file__)]
    if _stale(TORCH_OUT, deps) or not os.path.exists(TORCH_STAMP):
        return True
    with open(TORCH_STAMP) as f:
        return f.read() != version


def _build_torch(force):
    version = _torch_version()
    if version is None:  # the C library and its binding need no torch
        return
    if not force and not _torch_stale(version):
        return
    import torch
    from torch.utils import cpp_extension
    include = ["-isystem" + p for p in cpp_extension.include_paths() + [sysconfig.get_paths()["include"],
                                                                        os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = TORCH_OUT + ".tmp%d" % os.getpid()
    # libkd.so is found beside the module, torch's libraries where torch has loaded them
    subprocess.check_call([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
                           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
                           "-I" + os.path.join(ROOT, "include"), *include, TORCH_SOURCE, "-o", tmp, "-L" + HERE, "-l:libkd.so",
                           "-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                           "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, TORCH_OUT)
    os.makedirs(os.path.dirname(TORCH_STAMP), exist_ok=True)
    with open(TORCH_STAMP, "w") as f:
        f.write(version)


def build(force: bool = False, verbose: bool = False) -> str:
    _build_lib(force, verbose)
    _build_torch(force)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
