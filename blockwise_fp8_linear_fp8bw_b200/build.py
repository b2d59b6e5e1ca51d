"""Build the CUDA library libfp8bw.so in-tree for sm_100a (nvcc, no torch), and
its Python binding.

Two translation units, each including its kernel headers: csrc/api.cu (the
quantisers and GEMMs) and csrc/layer/layer.cu (the operators around them);
cudart is linked statically; the driver's TMA encoder is reached through
cudaGetDriverEntryPoint, so no libcuda link is needed at build time. Besides,
one CPython extension module (csrc/layer/binding.cpp, host code) that gives the
layer operators' Python calls a short path.
"""
import importlib.metadata
import os
import subprocess
import sys
import sysconfig

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


# The Python binding of the layer operators: a CPython extension module, host
# code only, compiled against the installed torch. It calls the library through the
# header's types and torch through its C++ interface, so either one's change rebuilds
# it; the torch version it was compiled for stands in the module.
BINDING_SRC = os.path.join(CSRC, "layer", "binding.cpp")
BINDING = os.path.join(HERE, "_layer_binding" + sysconfig.get_config_var("EXT_SUFFIX"))


def _torch_version():
    """The installed torch's version (without importing it), or None."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None


def _binding_stale() -> bool:
    version = _torch_version()
    if version is None:          # nothing to bind to: the library is all there is
        return False
    if not os.path.exists(BINDING):
        return True
    t = os.path.getmtime(BINDING)
    if any(os.path.getmtime(s) > t for s in (BINDING_SRC, HEADER, LAYER_HEADER)):
        return True
    with open(BINDING, "rb") as fh:
        return ("fp8bw binding for torch %s\0" % version).encode() not in fh.read()


def build_binding(force: bool = False) -> str:
    if not force and not _binding_stale():
        return BINDING
    import torch
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    tmp = BINDING + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           '-DFP8BW_TORCH_VERSION="%s"' % _torch_version(),
           "-I" + os.path.join(root, "include"),
           "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"),
           "-o", tmp, BINDING_SRC, "-L" + lib, "-Wl,-rpath," + lib,
           "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("g++ failed building the layer operators' binding")
    os.replace(tmp, BINDING)
    return BINDING


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or
                     not os.path.isabs(cand)):
            return cand
    return "nvcc"


def needs_build() -> bool:
    return _lib_stale() or _binding_stale()


def _lib_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in _sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if force or _lib_stale():
        _build_lib(verbose)
    if _torch_version() is not None:
        build_binding(force)
    return LIB


def _build_lib(verbose: bool) -> None:
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


if __name__ == "__main__":
    print(build(force=True, verbose=True))
