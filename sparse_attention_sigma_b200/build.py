"""Build the CUDA library ``libhad.so`` in-tree for sm_100a (B200).

``nvcc`` cross-compiles without a GPU.  The library links the CUDA runtime
statically, so it only needs the driver at run time.  Fast-math is off on
purpose: the standardize step relies on IEEE division with subnormals.
"""
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libhad.so")
SOURCES = ["had_api.cu", "had_cache.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler",
         "-fvisibility=hidden", "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _newest_input():
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return max(os.path.getmtime(p) for p in paths)


def build(force: bool = False, verbose: bool = False) -> str:
    if (not force and os.path.exists(LIB)
            and os.path.getmtime(LIB) >= _newest_input()):
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
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
