"""Builds libidx.so in-tree: nvcc for sm_103a, one object per translation unit
compiled in parallel, then a shared-library link; and _serve.so, the serving
operators' Python binding (host C++ against PyTorch), again for every PyTorch.  Without
PyTorch only libidx.so is built.  No GPU is needed to build."""
from __future__ import annotations

import glob
import importlib.metadata
import os
import platform
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libidx.so")
BINDING = os.path.join(CSRC, "serve_binding.cpp")
BINDING_LIB = os.path.join(OUT_DIR, "_serve.so")
TAG = ".for"  # suffix of the file that names the PyTorch of a binding
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _fresh(out: str, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps)


def _lib_fresh() -> bool:
    headers = [os.path.join(CSRC, "*.cuh"), os.path.join(CSRC, "*.h"), os.path.join(INCLUDE, "*.h")]
    return _fresh(LIB, sources() + [f for h in headers for f in glob.glob(h)])


def torch_tag() -> str | None:
    """The PyTorch and Python that a binding is for; None where there is no PyTorch."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None
    return f"torch {version} {sys.implementation.cache_tag} {platform.machine()}"


def _binding_fresh(tag: str | None) -> bool:
    if tag is None:
        return True  # nothing to bind to: only the C library is built
    if not _fresh(BINDING_LIB, [BINDING, os.path.join(INCLUDE, "idx.h")]):
        return False
    try:
        with open(BINDING_LIB + TAG) as f:
            return f.read() == tag
    except OSError:
        return False


def up_to_date() -> bool:
    return _lib_fresh() and _binding_fresh(torch_tag())


def _binding_command(out: str):
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    includes = [os.path.join(root, "include"),
                os.path.join(root, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    lib = os.path.join(root, "lib")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
            *(a for i in includes for a in ("-isystem", i)), BINDING, "-o", out, f"-L{lib}",
            f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None,
          out_dir: str | None = None) -> str:
    """Builds what is missing or older than its sources; the path of libidx.so."""
    out_dir = out_dir or OUT_DIR
    in_tree = out_dir == OUT_DIR
    tag = torch_tag()
    lib_needed = force or not in_tree or not _lib_fresh()
    binding_needed = tag is not None and (force or not in_tree or not _binding_fresh(tag))
    os.makedirs(out_dir, exist_ok=True)
    binding = os.path.join(out_dir, "_serve.so")
    with ThreadPoolExecutor(max_workers=1) as ex:
        bound = ex.submit(_build_binding, binding, tag) if binding_needed else None
        if lib_needed:
            _build_lib(os.path.join(out_dir, "libidx.so"), verbose, extra or [])
        if bound:
            bound.result()
    return os.path.join(out_dir, "libidx.so")


def _build_lib(lib: str, verbose: bool, extra: list[str]):
    nvcc = _nvcc()
    flags = ARCH + NVCC_FLAGS + extra

    def compile_one(src):
        obj = os.path.join(os.path.dirname(lib), os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        results = list(ex.map(compile_one, sources()))
    errors = [(s, r) for s, _, r in results if r.returncode != 0]
    for s, _, r in results:
        if verbose or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
    if errors:
        raise RuntimeError("nvcc failed for: " + ", ".join(os.path.basename(s) for s, _ in errors))
    tmp = lib + f".{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for _, o, _ in results], "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link of libidx.so failed")
    os.replace(tmp, lib)


def _build_binding(out: str, tag: str):
    tmp = out + f".{os.getpid()}.tmp"
    r = subprocess.run(_binding_command(tmp), capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("build of the serving operators' binding failed")
    os.replace(tmp, out)
    with open(out + TAG, "w") as f:
        f.write(tag)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
