"""Build the CUDA library libfp8bw.so in-tree for sm_100a (nvcc, no torch).

Two translation units, each including its kernel headers: csrc/api.cu (the
quantisers and GEMMs) and csrc/layer/layer.cu (the operators around them);
cudart is linked statically; the driver's TMA encoder is reached through
cudaGetDriverEntryPoint, so no libcuda link is needed at build time.
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfp8bw.so")
ROOT = os.path.dirname(HERE)
HEADER = os.path.join(ROOT, "include", "fp8bw.h")
LAYER_HEADER = os.path.join(ROOT, "include", "fp8bw_layer.h")
UNITS = [os.path.join(CSRC, "api.cu"), os.path.join(CSRC, "layer", "layer.cu")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-Xptxas", "-v", "--threads", "2",
]


def _sources():
    srcs = [os.path.join(d, f) for d in (CSRC, os.path.join(CSRC, "layer"))
            for f in sorted(os.listdir(d)) if f.endswith((".cu", ".cuh"))]
    return srcs + [HEADER, LAYER_HEADER]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or
                     not os.path.isabs(cand)):
            return cand
    return "nvcc"


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in _sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [_nvcc()] + NVCC_FLAGS + ["-o", tmp] + UNITS
    res = subprocess.run(cmd, capture_output=True, text=True)
    log = res.stdout + res.stderr
    with open(os.path.join(HERE, "build.log"), "w") as fh:
        fh.write(" ".join(cmd) + "\n" + log)
    if res.returncode != 0:
        sys.stderr.write(log)
        raise RuntimeError("nvcc failed building libfp8bw.so")
    if verbose:
        sys.stdout.write(log)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
