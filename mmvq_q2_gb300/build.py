"""Build libq2k.so in-tree with nvcc for sm_103a (no cmake, no torch), and
the binding's native half with the host's C compiler and Python's headers.

Usage: ``python -m mmvq_q2_gb300.build`` or ``build()`` from Python.  The
translation units compile in parallel; the shared library lands in
``mmvq_q2_gb300/_lib/libq2k.so``, the extension module beside it.  Where there
is no Python.h or no host C compiler the library is built all the same, and
the Python calls that need the extension module say so.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shlex
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT, "libq2k.so")
SOURCES = ["q2k_api.cu", "q2k_mv.cu", "q2k_m1.cu", "q2k_mmq.cu", "q2k_mt.cu", "q2k_small.cu", "q2k_gemm.cu", "q2k_umma.cu", "q3k_mv.cu", "q3k_mt.cu",
           "kv_page.cu", "kv_attn.cu", "layer_ops.cu", "fp8_ops.cu", "fp8_gemm.cu", "fp8_stream.cu"]
CALLS_SOURCE = "q2k_python.c"
CALLS = os.path.join(OUT, "_q2kcall" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
                   "-Xptxas", "-warn-spills"] + list(extra)


def host_cc():
    """The host's C compiler as a list of words ($CC may have arguments), None without one."""
    cc = shlex.split(os.environ.get("CC", "")) or [shutil.which("gcc") or shutil.which("cc")]
    return cc if cc[0] else None


def _no_calls() -> str:
    """Why the extension module cannot be built here; empty where it can."""
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        return f"no Python.h in {include}"
    return "" if host_cc() else "no host C compiler"


def _up_to_date() -> bool:
    built = [LIB] + ([] if _no_calls() and not os.path.exists(CALLS) else [CALLS])
    if not all(os.path.exists(f) for f in built):
        return False
    t = min(os.path.getmtime(f) for f in built)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(os.path.dirname(HERE), "include", "q2k.h"))
    return all(os.path.getmtime(d) <= t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and _up_to_date():
        return LIB
    os.makedirs(OUT, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(OUT, src.replace(".cu", ".o"))
        cmd = [cc, *_flags(extra_flags), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    def compile_calls():
        why = _no_calls()
        if why:
            if os.path.exists(CALLS):  # of older sources
                os.remove(CALLS)
            print(f"{os.path.basename(CALLS)} is not built ({why}): the decode-layer calls of the Python binding need it",
                  file=sys.stderr)
            return
        tmp = CALLS + f".{os.getpid()}.tmp"
        host = host_cc()
        cmd = [*host, "-O2", "-std=c11", "-Wall", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"],
               os.path.join(CSRC, CALLS_SOURCE), "-o", tmp, "-lm"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{host[0]} failed on {CALLS_SOURCE}:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, CALLS)

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(compile_calls)
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for obj, err in results:
            if err.strip():
                print(err, file=sys.stderr)
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    calls.result()  # the library does not depend on it
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
