"""Builds libfa.so in-tree with nvcc for sm_103a.

The library is two translation units that include their kernels, compiled at
once: ``csrc/fa_api.cu`` (attention forward) and ``csrc/fa_serve.cu`` (paged
cache and rotary positions). It links the CUDA runtime statically and resolves
the driver's tensor-map encoder at run time, so it needs no libcuda at link
time.

The Python binding's native half (``csrc/fa_bind.cpp``, torch's C++ API) is
compiled beside it with the host compiler into ``lib/_fa_bind-torch<version>.so``
and linked to libfa.so.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libfa.so")


def bind_path() -> str:
    """The binding's native half, named after the torch that it is built for
    (another torch's C++ API may differ)."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "none"
    return os.path.join(LIB_DIR, f"_fa_bind-torch{version}.so")


BIND_PATH = bind_path()
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc_path() -> str:
    cuda_home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda_home, "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or cand)


def sources() -> list[str]:
    out = []
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h", ".cpp")):
            out.append(os.path.join(CSRC, name))
    out.append(os.path.join(INCLUDE, "fa.h"))
    return out


def nvcc_cmd(out_path: str, extra: list[str] | None = None) -> list[str]:
    return [nvcc_path(), ARCH, "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
            "-Xcompiler", "-fPIC", "-shared", "--threads", "2", "-I", INCLUDE, "-I", CSRC,
            *(extra or []), os.path.join(CSRC, "fa_api.cu"), os.path.join(CSRC, "fa_serve.cu"), "-o", out_path]


def bind_cmds(obj: str, out_path: str) -> tuple[list[str], list[str]]:
    """Compile and link commands of the binding's native half."""
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda_home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cxx = os.environ.get("CXX", "g++")
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-c", "-I", INCLUDE, "-isystem", os.path.join(torch_dir, "include"),
                "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda_home, "include"),
                os.path.join(CSRC, "fa_bind.cpp"), "-o", obj]
    link = [cxx, "-shared", obj, "-o", out_path, "-L", LIB_DIR, "-l:libfa.so", "-L", os.path.join(torch_dir, "lib"),
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def up_to_date() -> bool:
    if not (os.path.exists(LIB_PATH) and os.path.exists(BIND_PATH)):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BIND_PATH))
    return all(os.path.getmtime(s) <= t for s in sources())


# Kernels that split registers between warpgroups with setmaxnreg: the split
# in the source assumes this many registers per thread at launch (384 threads
# x 168). A different count would make setmaxnreg.inc wait for registers that
# never come, so the build refuses it.
LAUNCH_REGS = {"fa_fwd_kernel": 168}


def check_ptxas_report(report: str) -> dict[str, int]:
    """Parses `ptxas -v` output into {kernel: registers} and enforces LAUNCH_REGS."""
    regs, current = {}, None
    for line in report.splitlines():
        m = re.search(r"Compiling entry function '([^']+)'", line)
        if m:
            current = m.group(1)
            continue
        m = re.search(r"Used (\d+) registers", line)
        if m and current:
            regs[current] = int(m.group(1))
            current = None
    for name in LAUNCH_REGS:
        if not any(name in mangled for mangled in regs):
            raise RuntimeError(f"ptxas report lists no register count for {name}")
    for mangled, n in regs.items():
        for name, want in LAUNCH_REGS.items():
            if name in mangled and n != want:
                raise RuntimeError(f"{mangled}: ptxas allocated {n} registers per thread, the register "
                                   f"split assumes {want}")
    return regs


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile libfa.so and the binding if any source is newer than them.
    Returns the path of libfa.so."""
    if not force and not extra and up_to_date():
        return LIB_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp, obj, tmp_bind = (f"{path}.tmp{os.getpid()}" for path in (LIB_PATH, BIND_PATH + ".o", BIND_PATH))
    cmd = nvcc_cmd(tmp, ["-Xptxas", "-v"] + (extra or []))
    compile_bind, link_bind = bind_cmds(obj, tmp_bind)
    try:
        with subprocess.Popen(compile_bind, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) as bind:
            res = subprocess.run(cmd, capture_output=True, text=True)
            bind_report = bind.communicate()[0]
        if verbose or res.returncode != 0:
            sys.stderr.write(res.stdout + res.stderr)
        if res.returncode != 0:
            raise subprocess.CalledProcessError(res.returncode, cmd)
        check_ptxas_report(res.stdout + res.stderr)
        if bind.returncode != 0:
            sys.stderr.write(bind_report)
            raise subprocess.CalledProcessError(bind.returncode, compile_bind)
        os.replace(tmp, LIB_PATH)
        subprocess.run(link_bind, check=True)
        os.replace(tmp_bind, BIND_PATH)
    finally:
        for path in (tmp, obj, tmp_bind):
            if os.path.exists(path):
                os.remove(path)
    return LIB_PATH


if __name__ == "__main__":  # pragma: no cover
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
