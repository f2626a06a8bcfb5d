"""Build the sm_100a shared library libgemm_epi.so in the package directory.

    python -m activation_epilogue_tcgen05_b200.build [--force] [-j N]

Every ``csrc/*.cu`` file is compiled with nvcc for ``sm_100a`` (in parallel,
incrementally: an object is rebuilt when its source or any ``csrc`` header or
``include/gemm_epi.h`` is newer) and linked with the static CUDA runtime, so
the library needs only the NVIDIA driver at run time.  The driver API
(tensor-map encoding) is reached through ``cudaGetDriverEntryPoint``; nothing
links libcuda directly, so the library also loads on machines without a GPU
(where every entry point that needs a device returns GEMM_EPI_ERR_NO_DEVICE).

Beside it, ``binding/operands.cpp`` becomes ``_operands.so`` (g++, torch's headers): the Python binding's checks of operands,
compiled.  Where that cannot be built the binding's own Python forms are used, and the build says so.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import contextlib
import glob
import json
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgemm_epi.so")

OPERANDS = os.path.join(PKG, "binding", "operands.cpp")
OPERANDS_SO = os.path.join(PKG, "_operands.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(INCLUDE, "gemm_epi.h")]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, obj, verbose):
    cmd = [nvcc()] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj


def source_hash() -> str:
    """sha1 over every source, header and compiler flag that goes into the library."""
    import hashlib
    h = hashlib.sha1(" ".join(ARCH + NVCC_FLAGS[:-4]).encode())
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + _headers()):
        with open(path, "rb") as f:
            h.update(os.path.basename(path).encode())
            h.update(f.read())
    return h.hexdigest()


def _compile_operands(out, verbose):
    import torch
    at = os.path.dirname(torch.__file__)
    include = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), sysconfig.get_paths()["include"]]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f"-DBUILT_FOR={json.dumps(f'{torch.__version__} {sys.version}')}",
           OPERANDS, "-o", out]
    cmd += [a for i in include for a in ("-isystem", i)]
    cmd += ["-L" + os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(r.stderr[-2000:])


def build_operands(force: bool = False, verbose: bool = False) -> bool:
    """Compile (if stale) the binding's operand checks; whether they are there.  Without torch, a C++ compiler or a folder to write
    to they are not (nor is a stale module, then), which is no error."""
    import hashlib
    import importlib.metadata
    stamp, tmp = OPERANDS_SO + ".sha1", OPERANDS_SO + f".tmp{os.getpid()}"
    try:
        with open(OPERANDS, "rb") as f:
            digest = hashlib.sha1(f.read() + f"{importlib.metadata.version('torch')} {sys.version}".encode()).hexdigest()
        if not force and os.path.exists(OPERANDS_SO) and os.path.exists(stamp):
            with open(stamp) as f:
                if f.read().strip() == digest:
                    return True
        _compile_operands(tmp, verbose)
        os.replace(tmp, OPERANDS_SO)
        with open(stamp, "w") as f:
            f.write(digest + "\n")
    except (ImportError, OSError, RuntimeError) as e:
        print(f"{os.path.basename(OPERANDS)} was not built; the binding checks its operands in Python:\n{e}", file=sys.stderr)
        with contextlib.suppress(OSError):
            os.remove(OPERANDS_SO)
        return False
    return True


def build(force: bool = False, jobs: int | None = None, verbose: bool = False) -> str:
    """Compile (if stale) and link libgemm_epi.so, and the binding's operand checks; return the library's path.

    The library is current when its stamp file holds the hash of the present
    sources (copies that do not keep file times stay current)."""
    build_operands(force, verbose)
    stamp = LIB + ".sha1"
    digest = source_hash()
    if not force and os.path.exists(LIB) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == digest:
                return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdrs = _headers()
    objs, todo = [], []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            todo.append((s, o))
    if todo:
        jobs = jobs or min(len(todo), os.cpu_count() or 4)
        with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
            for f in [ex.submit(_compile, s, o, verbose) for s, o in todo]:
                f.result()
    if force or todo or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs + ["-lpthread", "-ldl", "-lrt"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    with open(stamp, "w") as f:
        f.write(digest + "\n")
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-j", "--jobs", type=int, default=None)
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(a.force, a.jobs, a.verbose))


if __name__ == "__main__":
    sys.exit(main())
