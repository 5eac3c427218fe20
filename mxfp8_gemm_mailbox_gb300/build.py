"""Build ``libmxfp8_mailbox.so`` in-tree with nvcc for sm_103a, and the Python
module ``_calls`` over it with the host compiler.

The translation units compile in parallel (one ``-gencode``), then link into
one shared library and the module next to this file.  Run ``python -m
mxfp8_gemm_mailbox_gb300.build`` or call :func:`build`.
"""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from pathlib import Path

PACKAGE = Path(__file__).resolve().parent
ROOT = PACKAGE.parent
CSRC = PACKAGE / "csrc"
INCLUDE = ROOT / "include"
BUILD_DIR = PACKAGE / "_build"
LIBRARY = PACKAGE / "libmxfp8_mailbox.so"
SOURCES = ("publish_gemm.cu", "publish_gemm_fold.cu", "publish_gemm_k256.cu", "mailbox.cu",
           "lamport_gather.cu", "tagged_mailbox.cu", "adapters.cu", "latent_project.cu",
           "latent_attend.cu", "abi_latent.cu", "experts_route.cu", "quantize.cu",
           "experts_product.cu", "abi_experts.cu", "abi.cu")
CALLS = PACKAGE / ("_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _stale() -> bool:
    if not LIBRARY.exists() or not CALLS.exists():
        return True
    newest = max(p.stat().st_mtime for p in list(CSRC.iterdir()) + list(INCLUDE.iterdir()))
    return min(LIBRARY.stat().st_mtime, CALLS.stat().st_mtime) < newest


def _compile_calls(nvcc: str) -> Path:
    """``csrc/calls.cpp``, against this interpreter's and torch's headers."""
    obj = BUILD_DIR / "calls.o"
    torch = Path(importlib.util.find_spec("torch").origin).parent / "include"
    includes = [INCLUDE, torch, torch / "torch/csrc/api/include",
                sysconfig.get_paths()["include"], Path(nvcc).resolve().parents[1] / "include"]
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-w",
          *(f"-I{i}" for i in includes), "-c", str(CSRC / "calls.cpp"), "-o", str(obj)],
         "compiling calls.cpp")
    return obj


def _run(cmd: list, what: str) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stdout}\n{res.stderr}")


def _link_calls(obj: Path) -> None:
    """The module next to the library it calls."""
    lib = Path(importlib.util.find_spec("torch").origin).parent / "lib"
    tmp = CALLS.with_suffix(f".{os.getpid()}.tmp")
    _run([os.environ.get("CXX", "g++"), "-shared", str(obj), "-o", str(tmp), f"-L{PACKAGE}",
          f"-l:{LIBRARY.name}", "-Wl,-rpath,$ORIGIN", f"-L{lib}", "-ltorch_python", "-ltorch_cpu",
          "-lc10", "-lc10_cuda"], "linking _calls")
    os.replace(tmp, CALLS)


def build(force: bool = False, verbose: bool = False) -> Path:
    """Compile the CUDA library if a source is newer than it (or ``force``)."""
    if not force and not _stale():
        return LIBRARY
    nvcc = _nvcc()
    BUILD_DIR.mkdir(exist_ok=True)
    common = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              f"-I{INCLUDE}", f"-I{CSRC}"]
    if verbose:
        common.append("-Xptxas=-v")

    def compile_one(name: str) -> Path:
        obj = BUILD_DIR / (name + ".o")
        cmd = [*common, "-c", str(CSRC / name), "-o", str(obj)]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {name}:\n{res.stdout}\n{res.stderr}")
        if verbose and res.stderr:
            sys.stderr.write(res.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as pool:
        calls = pool.submit(_compile_calls, nvcc)
        objs = list(pool.map(compile_one, SOURCES))
        calls_obj = calls.result()
    tmp = LIBRARY.with_suffix(f".{os.getpid()}.tmp")
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", *map(str, objs), "-o", str(tmp)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"linking failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIBRARY)
    _link_calls(calls_obj)
    return LIBRARY


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIBRARY)
