"""Build ``libpa.so`` (the C ABI of ``include/pa.h``) in-tree for sm_103a.

Each translation unit is compiled by nvcc in parallel, then linked into one
shared library with the CUDA runtime linked statically.  Beside it, ``_marshal``
(``csrc/marshal.cpp``), the Python extension that passes torch tensors to some
of its functions, is compiled by g++ against the installed torch and Python;
where that cannot be done it is left out, with a word about it, and the calls
take the longer way through ctypes.  Only sources or headers newer than their object are rebuilt.  Run ``python -m
paged_kv_cache_76_gb300.build [--force] [--verbose]``.
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpa.so")
SOURCES = ["pa_api.cu", "decode.cu", "prefill.cu", "cache_ops.cu", "block_alloc.cpp", "decode_noalloc.cu", "attn_tc.cu",
           "attn_tile.cu", "vkv.cpp", "rope.cu", "evict.cu", "tree.cu", "pa_kv4.cu", "kv4_cache.cu", "kv4_decode.cu",
           "kv4_prefill.cu", "fork.cu"]
MARSHAL = os.path.join(HERE, "_marshal" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
MARSHAL_STAMP = os.path.join(OBJDIR, "marshal.stamp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpa.so")


def _headers():
    hs = [os.path.join(INCLUDE, "pa.h")]
    hs += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return hs


def _stale(obj: str, deps) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_version(torch_dir: str):
    """torch.__version__ without importing torch; None if it is not where it always is."""
    try:
        with open(os.path.join(torch_dir, "version.py")) as f:
            m = re.search(r"""^__version__ = ['"](.+)['"]$""", f.read(), re.M)
    except OSError:
        return None
    return m and m.group(1)


def _marshal_job(nvcc: str):
    """(command up to the output's name, stamp) that compiles _marshal, or a text: why it cannot be."""
    spec = importlib.util.find_spec("torch")
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    if spec is None or not spec.submodule_search_locations:
        return "torch is not installed"
    if cxx is None:
        return "there is no C++ compiler"
    torch_dir = spec.submodule_search_locations[0]
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
           os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")]
    if not os.path.exists(os.path.join(inc[1], "Python.h")) or not os.path.isdir(inc[2]):
        return "torch's or Python's headers are missing"
    version = _torch_version(torch_dir)
    if version is None:
        return "torch's version is not known"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared"] + [x for i in inc for x in ("-I", i)]
    cmd += [f'-DPA_TORCH_VERSION="{version}"', os.path.join(CSRC, "marshal.cpp"), "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu",
            "-lc10", "-lc10_cuda", "-o"]
    # built for one torch and one Python: another of either is another build
    return cmd, f"torch {version} python {sys.version}"


def _marshal_fresh(stamp: str) -> bool:
    try:
        with open(MARSHAL_STAMP) as f:
            same = f.read() == stamp
    except OSError:
        return False
    return same and not _stale(MARSHAL, [os.path.join(CSRC, "marshal.cpp"), os.path.join(INCLUDE, "pa.h")])


def _remove(*paths) -> None:
    for p in paths:
        if os.path.exists(p):
            os.remove(p)


def _build_marshal(nvcc: str, force: bool, verbose: bool) -> None:
    """Compile _marshal if it is not up to date.  It is optional: where that fails it is left out, an older one too."""
    job = _marshal_job(nvcc)
    if not isinstance(job, str):
        cmd, stamp = job
        if not force and _marshal_fresh(stamp):
            return
        new = MARSHAL + f".{os.getpid()}.tmp"
        r = subprocess.run(cmd + [new], capture_output=True, text=True)
        if verbose or r.returncode:
            sys.stderr.write(" ".join(cmd + [new]) + "\n" + r.stdout + r.stderr)
        if r.returncode == 0:
            os.replace(new, MARSHAL)
            with open(MARSHAL_STAMP, "w") as f:
                f.write(stamp)
            return
        _remove(new)
        job = "its compilation failed"
    _remove(MARSHAL, MARSHAL_STAMP)
    sys.stderr.write(f"_marshal is left out ({job}): its calls go through ctypes\n")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link; returns the path of libpa.so."""
    nvcc = _nvcc()
    os.makedirs(OBJDIR, exist_ok=True)
    headers = _headers()
    common = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    jobs = []
    objs = []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(OBJDIR, src + ".o")
        objs.append(obj)
        if force or _stale(obj, [path] + headers):
            cmd = [nvcc] + common + ["-c", path, "-o", obj]
            if src.endswith(".cu"):
                cmd[1:1] = ARCH + ["-lineinfo"]
                if verbose:
                    cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 4)) as ex:
        marshal = ex.submit(_build_marshal, nvcc, force, verbose)
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode:
                raise RuntimeError("nvcc failed on " + next(a for a in cmd if a.startswith(CSRC + os.sep)))
        marshal.result()
    if force or jobs or _stale(LIB, objs):
        cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", LIB] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            raise RuntimeError("link of libpa.so failed")
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print nvcc commands and ptxas register usage")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    main()
