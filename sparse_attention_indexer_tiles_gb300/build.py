"""Builds libidx.so in-tree: nvcc for sm_103a, one object per translation unit
compiled in parallel, then a shared-library link; and _serve.so, the serving
operators' Python binding (host C++ against PyTorch).  No GPU is needed to build."""
from __future__ import annotations

import glob
import os
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


def _deps():
    headers = [os.path.join(CSRC, "*.cuh"), os.path.join(CSRC, "*.h"), os.path.join(INCLUDE, "*.h")]
    return sources() + [BINDING] + [f for h in headers for f in glob.glob(h)]


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(BINDING_LIB)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING_LIB))
    return all(os.path.getmtime(p) <= t for p in _deps())


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
    out_dir = out_dir or OUT_DIR
    lib = os.path.join(out_dir, "libidx.so")
    if not force and out_dir == OUT_DIR and up_to_date():
        return LIB
    os.makedirs(out_dir, exist_ok=True)
    nvcc = _nvcc()
    flags = ARCH + NVCC_FLAGS + (extra or [])

    def compile_one(src):
        obj = os.path.join(out_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    binding = os.path.join(out_dir, "_serve.so")
    binding_tmp = binding + f".{os.getpid()}.tmp"

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        bound = ex.submit(lambda: subprocess.run(_binding_command(binding_tmp),
                                                 capture_output=True, text=True))
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
    r = bound.result()
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("build of the serving operators' binding failed")
    os.replace(binding_tmp, binding)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
