"""Builds libspecverify.so in-tree with nvcc for sm_103a (GB300), and beside it
the argument side of the drafted tree's operators, a Python extension on torch's
tensors, with g++."""

from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
import warnings

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
INCLUDE = os.path.join(ROOT, "include")
SOURCES = [os.path.join(PKG_DIR, "csrc", name)
           for name in ("specverify.cu", "cache.cu", "attention.cu", "logits.cu", "beams.cu",
                        "chunk.cu", "chunk_bf16.cu", "chunk_f16.cu")]
HEADERS = [os.path.join(INCLUDE, "specverify.h"),
           *(os.path.join(PKG_DIR, "csrc", name) for name in ("cache.cuh", "tensor.cuh", "chunk.cuh", "single.cuh"))]
LIB_PATH = os.path.join(PKG_DIR, "libspecverify.so")
BINDING_SOURCE = os.path.join(PKG_DIR, "csrc", "binding.cpp")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecverify")


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def binding_path() -> str:
    """The extension's file: one of another torch or Python does not load, so both
    versions are in its name."""
    import torch
    return os.path.join(
        PKG_DIR, f"_binding-{torch.__version__}-py{sysconfig.get_python_version()}.so")


_binding_failure = None


def binding_failure():
    """Why this process's build() left the extension unbuilt, or None."""
    return _binding_failure


def _keep_failure(why: str):
    global _binding_failure
    _binding_failure = why
    if os.path.exists(binding_path()):  # of an older source: not to be loaded for this one
        os.remove(binding_path())
    warnings.warn(f"the library is built without the drafted tree's operators in Python: {why}")


def _build_binding(force: bool, verbose: bool):
    """Starts the extension's compiler where it is needed; returns what waits for
    it.  Without torch there are no tensors to bind and nothing is built; where it cannot
    be built, the reason is kept for the calls that need it."""
    global _binding_failure
    try:
        import torch
    except ImportError:
        return lambda: None
    home = os.path.dirname(torch.__file__)
    path = binding_path()
    if not force and not _stale(path, [BINDING_SOURCE, HEADERS[0]]):
        _binding_failure = None
        return lambda: None
    if torch.version.cuda is None:
        return lambda: _keep_failure("this torch has no CUDA")
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    include = [INCLUDE, os.path.join(home, "include"),
               os.path.join(home, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in include), BINDING_SOURCE, "-o", tmp, f"-L{home}/lib",
           f"-Wl,-rpath,{home}/lib", "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd))
    try:
        compiler = subprocess.Popen(cmd, stderr=subprocess.PIPE, text=True)
    except OSError as e:
        why = str(e)
        return lambda: _keep_failure(why)

    def wait():
        global _binding_failure
        said = compiler.communicate()[1]
        if compiler.returncode != 0:
            _keep_failure(f"{cmd[0]} failed: {said[-4000:]}")
            return
        os.replace(tmp, path)
        _binding_failure = None
    return wait


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile the CUDA library and the binding's extension where a source or
    header is newer than them.  An extension that cannot be built is a warning: the
    library stands without it."""
    wait = _build_binding(force, verbose)
    try:
        _build_library(force, verbose, extra_flags)
    finally:
        wait()
    return LIB_PATH


def _build_library(force: bool, verbose: bool, extra_flags):
    if not force and not _stale(LIB_PATH, SOURCES + HEADERS):
        return
    nvcc = nvcc_path()
    cuda_lib = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-I", INCLUDE,
           "-shared", "-Xcompiler", "-fPIC", "-cudart", "shared", "--threads", str(len(SOURCES)),
           "-Xlinker", f"-rpath,{cuda_lib}", *extra_flags, "-o", tmp, *SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    print(build(force=True, verbose=True))
