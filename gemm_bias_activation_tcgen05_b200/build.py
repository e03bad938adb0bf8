"""Build the sm_100a shared library ``libfused_linear.so`` in-tree with nvcc.

The library holds the C ABI of ``include/fused_linear.h`` and every CUDA
kernel of the fused linear layer.  It links the CUDA runtime statically and
reaches the driver's tensor-map encoder through the runtime's driver entry
point, so loading it needs no libcuda at link time.  Each source is compiled to
an object of its own, several at a time; an object whose sources have not changed
is kept.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libfused_linear.so")
OBJ_DIR = os.path.join(HERE, "_build")
_GEMM = ["fl_gemm.cuh", "fl_ptx.cuh", "fl_host.h"]
# each translation unit and the headers it includes
UNITS = {
    "fl_api.cu": ["fl_elementwise.cuh", "fl_plan.h", *_GEMM],
    "fl_pair.cu": ["fl_pair.cuh", "fl_plan.h", *_GEMM],
    "fl_small.cu": ["fl_small.cuh", "fl_pair.cuh", "fl_plan.h", *_GEMM],
    "fl_rows.cu": ["fl_rows.cuh", *_GEMM],
}
HEADER = os.path.join(ROOT, "include", "fused_linear.h")


def _src(name: str) -> str:
    return os.path.join(HERE, "csrc", name)


SOURCES = [_src(u) for u in UNITS]
DEPS = sorted({_src(f) for u, hs in UNITS.items() for f in (u, *hs)}) + [HEADER]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags():
    return ["-gencode", "arch=compute_100a,code=sm_100a", "-Xcompiler", "-fPIC", "-cudart", "static"]


def _object(unit: str) -> str:
    return os.path.join(OBJ_DIR, unit.replace(".cu", ".o"))


def compile_command(unit: str):
    return [nvcc(), *_flags(), "-lineinfo", "-O3", "-std=c++17", "-Xptxas", "-v",
            f"-I{os.path.join(ROOT, 'include')}", "-c", _src(unit), "-o", _object(unit)]


def link_command():
    return [nvcc(), *_flags(), "--shared", *[_object(u) for u in UNITS], "-o", LIB]


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def up_to_date() -> bool:
    return _newer(LIB, DEPS)


def _compile(unit: str, force: bool) -> str:
    """Compile one unit unless its object is current; its resource report (ptxas -v)."""
    report = _object(unit) + ".txt"
    deps = [_src(f) for f in (unit, *UNITS[unit])] + [HEADER]
    if not force and os.path.exists(report) and _newer(_object(unit), deps):
        return open(report).read()
    r = subprocess.run(compile_command(unit), capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"nvcc failed compiling {unit}")
    with open(report, "w") as f:
        f.write(r.stderr)
    return r.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(UNITS), os.cpu_count() or 1))) as ex:
        reports = list(ex.map(lambda u: _compile(u, force), UNITS))
    r = subprocess.run(link_command(), capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("nvcc failed linking libfused_linear.so")
    with open(os.path.join(HERE, "ptxas_report.txt"), "w") as f:
        f.write("".join(reports))
    if verbose:
        sys.stderr.write("".join(reports))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
