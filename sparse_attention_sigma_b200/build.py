"""Build the CUDA library ``libhad.so`` in-tree for sm_100a (B200), and the
Python module ``_cache.so`` that marshals the decoder cache's calls to it.

``nvcc`` cross-compiles without a GPU.  The library links the CUDA runtime
statically, so it only needs the driver at run time.  Fast-math is off on
purpose: the standardize step relies on IEEE division with subnormals.
"""
import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libhad.so")
BINDING = os.path.join(HERE, "_cache.so")
SOURCES = ["had_api.cu", "had_cache.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler",
         "-fvisibility=hidden", "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _newest_input():
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return max(os.path.getmtime(p) for p in paths)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and all(os.path.exists(f) and os.path.getmtime(f) >= _newest_input()
                         for f in (LIB, BINDING)):
        return LIB
    # one compiler per source, side by side, then the link
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, s + ".o") for s in SOURCES]
        jobs = [subprocess.Popen(["nvcc"] + ARCH + FLAGS + (["-Xptxas", "-v"] if verbose else []) +
                                 ["-c", os.path.join(CSRC, s), "-o", o])
                for s, o in zip(SOURCES, objects)]
        codes = [j.wait() for j in jobs]
        if any(codes):
            raise subprocess.CalledProcessError(next(c for c in codes if c), "nvcc")
        subprocess.run(["nvcc"] + ARCH + ["-shared", "-o", LIB + ".tmp"] + objects, check=True)
    os.replace(LIB + ".tmp", LIB)
    _build_binding()
    return LIB


def _build_binding():
    import sysconfig
    import torch
    home = os.path.dirname(os.path.abspath(torch.__file__))
    include = [os.path.join(home, "include"),
               os.path.join(home, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], INCLUDE, _cuda_include()]
    cmd = (["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] +
           [a for i in include for a in ("-isystem", i)] +
           [os.path.join(CSRC, "had_cache_bind.cpp"), "-o", BINDING + ".tmp",
            "-L", HERE, "-l:libhad.so", "-Wl,-rpath,$ORIGIN",
            "-L", os.path.join(home, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])
    subprocess.run(cmd, check=True)
    os.replace(BINDING + ".tmp", BINDING)


def _cuda_include():
    nvcc = shutil.which("nvcc")
    home = os.path.dirname(os.path.dirname(os.path.realpath(nvcc))) if nvcc else "/usr/local/cuda"
    return os.path.join(home, "include")


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
