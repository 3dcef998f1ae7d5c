"""Build libsa.so in-tree with nvcc for sm_103a.

Each CUDA translation unit compiles in its own nvcc process (in parallel),
then one link step makes ``stochastic_sliding_window_gb300/libsa.so``.
Beside it, with the host compiler, the serving calls' short way from Python
(``_paged_call.so``, against the installed torch): where that cannot be built
or loaded, the same calls go through ctypes.
Rebuilds only when a source or header is newer than the library.
"""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
BUILD = PKG / "_build"
LIB = PKG / "libsa.so"
CALL = PKG / "_paged_call.so"

SOURCES = ["sa_api.cu", "sa_perm.cu", "sa_simt.cu", "sa_tc.cu", "sa_tc_ring.cu", "sa_tc_chunk.cu",
           "sa_bwd.cu", "sa_graph.cu", "sa_prologue.cu", "sa_shard.cu", "sa_paged.cu",
           "sa_paged_rows.cu", "sa_paged_unit.cu", "sa_paged_tiles.cu",
           "sa_paged_order.cu", "sa_paged_members.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-v"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found")


def _inputs() -> list[Path]:
    return [CSRC / s for s in SOURCES] + list(CSRC.glob("*.cpp")) + list(CSRC.glob("*.h")) + list(CSRC.glob("*.cuh")) + \
        list(INCLUDE.glob("*.h")) + [Path(__file__)]


def up_to_date() -> bool:
    if not LIB.exists():
        return False
    t = LIB.stat().st_mtime
    return all(p.stat().st_mtime <= t for p in _inputs())


def _compile(src: str) -> tuple[str, str]:
    obj = BUILD / (Path(src).stem + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-I", str(INCLUDE), "-I", str(CSRC), "-c",
           str(CSRC / src), "-o", str(obj)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return str(obj), r.stderr


def _compile_call() -> str:
    """paged_call.cpp; returns what went wrong, if anything did."""
    CALL.unlink(missing_ok=True)
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return "torch is not installed"
    torch = Path(next(iter(spec.submodule_search_locations)))
    cuda = Path(nvcc()).resolve().parent.parent
    tmp = CALL.with_suffix(".so.tmp")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-w", "-I", str(INCLUDE),
           "-I", str(torch / "include"), "-I", str(torch / "include/torch/csrc/api/include"),
           "-I", sysconfig.get_path("include"), "-I", str(cuda / "include"), str(CSRC / "paged_call.cpp"),
           "-o", str(tmp), "-L", str(torch / "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
           "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        return r.stderr
    os.replace(tmp, CALL)
    return ""


def build(force: bool = False, verbose: bool = False) -> Path:
    """Compile and link libsa.so; returns its path."""
    if not force and up_to_date():
        return LIB
    BUILD.mkdir(exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        call = ex.submit(_compile_call)
        results = list(ex.map(_compile, SOURCES))
    if call.result():
        sys.stderr.write(f"paged_call.cpp not built, serving calls go through ctypes:\n{call.result()[-2000:]}\n")
    objs = [o for o, _ in results]
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB.with_suffix(".so.tmp")
    cmd = [nvcc(), *ARCH, "-shared", "-o", str(tmp), *objs, "-lcudart_static", "-lrt", "-ldl",
           "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
