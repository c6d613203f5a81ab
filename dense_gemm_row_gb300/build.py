"""Builds libdense_gemm_row.so in-tree from csrc/*.cu with nvcc for sm_103a.

Each translation unit is compiled in parallel to an object file under
``_build/``, then linked into a shared library with the CUDA runtime linked
statically, so the library needs no libcudart at load time and resolves the
driver only when a GPU call is made. Beside it, csrc/py_layers.cpp becomes the
Python module ``_layers`` (argument marshalling of the linear-layer operators;
needs the headers of Python and torch). Without torch the C library alone is
built; the module is built again when the Python or torch it was made for changes.

    python -m dense_gemm_row_gb300.build [--force] [--ptxas-verbose]
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB_NAME = "libdense_gemm_row.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
LAYERS_PATH = os.path.join(PKG, "_layers.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                     "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hdrs.append(os.path.join(INCLUDE, "dense_gemm_row.h"))
    return hdrs


def _torch_dir():
    """Directory of the torch package, or None without torch."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _layers_command(torch_dir: str, out: str):
    """g++ command that builds the _layers module against the running Python and torch."""
    import sysconfig
    inc = os.path.join(torch_dir, "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    return ["g++", "-O2", "-std=c++20", "-shared", "-fPIC", "-fvisibility=hidden", "-w",
            "-I", INCLUDE, "-isystem", inc,
            "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"],
            "-isystem", os.path.join(cuda, "include"),
            os.path.join(CSRC, "py_layers.cpp"), "-o", out,
            "-L", os.path.join(torch_dir, "lib"), "-Wl,-rpath," + os.path.join(torch_dir, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _layers_made_for(torch_dir: str) -> str:
    """What a built _layers module depends on beside its sources."""
    version = os.path.join(torch_dir, "version.py")
    return "\n".join([sys.version, sys.executable, torch_dir,
                      open(version).read() if os.path.exists(version) else ""])


def _stale(target: str, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(i) > t for i in inputs)


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = _sources()
    deps = _deps()
    objs = []
    jobs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src, *deps]):
            cmd = [cc, *NVCC_FLAGS, "-c", src, "-o", obj]
            if ptxas_verbose:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    # The _layers module needs torch; the C library does not, and is built without it.
    torch_dir = _torch_dir()
    layers_cmd = None
    layers_tmp, layers_stamp = LAYERS_PATH + f".tmp{os.getpid()}", os.path.join(BUILD, "layers.txt")
    if torch_dir is None:
        if not quiet:
            sys.stderr.write("torch not found: _layers (the linear-layer operators' Python "
                             "functions) is not built\n")
    else:
        made_for = _layers_made_for(torch_dir)
        if force or _stale(LAYERS_PATH, [os.path.join(CSRC, "py_layers.cpp"),
                                         os.path.join(INCLUDE, "dense_gemm_row.h")]) \
                or not os.path.exists(layers_stamp) or open(layers_stamp).read() != made_for:
            layers_cmd = _layers_command(torch_dir, layers_tmp)

    def run(cmd):
        return cmd, subprocess.run(cmd, capture_output=True, text=True)

    def check(cmd, res):
        if res.returncode != 0:
            raise RuntimeError("compiling failed:\n" + " ".join(cmd) + "\n" + res.stderr)
        if (ptxas_verbose or res.stderr.strip()) and not quiet:
            sys.stderr.write(res.stderr)

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 1))) as ex:
        layers = ex.submit(run, layers_cmd) if layers_cmd else None
        for cmd, res in ex.map(run, jobs):
            check(cmd, res)
    if force or jobs or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("link failed:\n" + " ".join(cmd) + "\n" + res.stderr)
        os.replace(tmp, LIB_PATH)
    if layers:  # behind the C library, which a failure here leaves in place
        check(*layers.result())
        os.replace(layers_tmp, LAYERS_PATH)
        with open(layers_stamp, "w") as f:
            f.write(made_for)
    return LIB_PATH


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_verbose=a.ptxas_verbose))
