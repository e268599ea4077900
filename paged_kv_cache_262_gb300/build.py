"""Builds libpagedattn in-tree: ``_build/libpagedattn.so`` for sm_103a.

Each translation unit is compiled in parallel (nvcc for ``.cu``, g++ for the
host-only ``.cpp``), then linked with nvcc into one shared library whose
exported symbols are the ``extern "C"`` calls of ``include/pagedattn.h``.

Where torch and its headers are there, the quick way into the long-context
calls (``fastcall/``, a CPython extension module) is built beside it; without
it those calls take their Python way.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
import threading
from typing import List, Optional

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libpagedattn.so")
INCLUDE = os.path.join(ROOT, "include")
FAST_SRC = os.path.join(HERE, "fastcall", "pa_fastcall.cpp")
FAST = os.path.join(OUT, "_pa_fastcall.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def sources() -> List[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "pagedattn.h"),
                                                                 __file__]
    return max(os.path.getmtime(f) for f in files)


def _fast_command(out: str) -> Optional[List[str]]:
    """The compile command of the extension module; None without torch."""
    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError:
        return None
    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"), INCLUDE]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-O2", "-std=c++20", "-fPIC", "-shared", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DPA_TORCH_VERSION="{torch.__version__}"', *[f"-I{i}" for i in inc], FAST_SRC,
            "-o", out, f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            f"-Wl,-rpath,{libs}"]


def _build_fast() -> None:
    """Builds the extension module if it is not up to date; a failure is
    reported and leaves the Python way."""
    deps = (FAST_SRC, os.path.join(INCLUDE, "pagedattn.h"), __file__)
    if os.path.exists(FAST) and os.path.getmtime(FAST) >= max(os.path.getmtime(f) for f in deps):
        return
    if os.path.exists(FAST):
        os.remove(FAST)
    tmp = FAST + f".tmp{os.getpid()}"
    cmd = _fast_command(tmp)
    if cmd is None:
        return
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        print(f"paged_kv_cache_262_gb300: the extension module was not built ({' '.join(cmd[:2])} ...):\n"
              f"{r.stderr[-2000:]}")
        return
    os.replace(tmp, FAST)


def build(force: bool = False, verbose: bool = False, extra_nvcc: List[str] = ()) -> str:
    os.makedirs(OUT, exist_ok=True)
    fast = threading.Thread(target=_build_fast)
    fast.start()
    try:
        return _build_lib(force, verbose, extra_nvcc)
    finally:
        fast.join()


def _build_lib(force: bool, verbose: bool, extra_nvcc: List[str]) -> str:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime():
        return LIB
    nvcc = _nvcc()
    common = ["-O3", "-std=c++17", "-I", INCLUDE, "-I", CSRC]
    jobs = []
    for src in sources():
        obj = os.path.join(OUT, os.path.basename(src) + ".o")
        if src.endswith(".cu"):
            cmd = [nvcc, *ARCH, "-lineinfo", *common, "-Xcompiler", "-fPIC", "-c", src, "-o", obj,
                   *extra_nvcc]
            if verbose:
                cmd += ["-Xptxas", "-v"]
        else:
            cuda_inc = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
            cmd = ["g++", *common, "-I", cuda_inc, "-fPIC", "-Wall", "-c", src, "-o", obj]
        jobs.append((cmd, obj))

    def run(job):
        cmd, obj = job
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
        logs = list(ex.map(run, jobs))
    if verbose:
        for l in logs:
            if l.strip():
                print(l)
    tmp = LIB + f".tmp{os.getpid()}"
    link = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for _, o in jobs], "-Xcompiler", "-fPIC"]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(link)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv))
