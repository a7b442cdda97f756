"""Builds the in-tree C-ABI library ``_build/libmx.so`` with nvcc for sm_103a.

Each CUDA translation unit compiles in parallel to an object file, then they
are linked into one shared library (static CUDA runtime, no libcuda link: the
driver entry point for tensor-map encoding is fetched at run time).  Beside it,
``_build/mx_torch.so``: the Python entry points of the operators between the
GEMMs (csrc/mx_torch.cpp, host code only, against the installed torch); where
torch is not installed the library alone is built, for users of its C ABI.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD_DIR, "libmx.so")
TORCH_SOURCE = "mx_torch.cpp"
TORCH_LIB = os.path.join(BUILD_DIR, "mx_torch.so")
TORCH_STAMP = TORCH_LIB + ".built_against"
# Bounds-checked variant (every kernel store guarded; see MX_ERR_BOUNDS in mx.h),
# used by the tests only.
CHECKED_DIR = os.path.join(HERE, "_build_checked")
CHECKED_LIB = os.path.join(CHECKED_DIR, "libmx.so")
SOURCES = ["mx_api.cu", "mx_quant.cu", "mx_gemm.cu", "mx_noalloc.cu", "mx_scales.cu",
           "mx_peak.cu", "mx_norm.cu", "mx_glu.cu", "mx_grad.cu", "mx_product.cu",
           "mx_act.cu", "mx_experts.cu", "mx_few.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the MXFP4 library needs the CUDA toolkit to build")
    return cand


def _deps() -> list[str]:
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    out.append(os.path.join(INCLUDE, "mx.h"))
    return out


def _stale(lib: str | None = None) -> bool:
    lib = lib or LIB
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in _deps())


def _torch_dir() -> str | None:
    """Folder of the installed torch; None without one."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None or spec.origin is None else os.path.dirname(spec.origin)


def _torch_stamp(torch: str) -> str:
    """What mx_torch.so is built against, beside the sources: Python, machine and torch."""
    with open(os.path.join(torch, "version.py")) as f:
        return "\n".join([str(sysconfig.get_config_var("SOABI")), torch, f.read()])


def fits_torch(torch: str | None = None) -> bool:
    """Whether mx_torch.so was built against this Python and the installed torch."""
    torch = torch or _torch_dir()
    if torch is None or not os.path.exists(TORCH_LIB) or not os.path.exists(TORCH_STAMP):
        return False
    with open(TORCH_STAMP) as f:
        return f.read() == _torch_stamp(torch)


def _compile_torch(torch: str, verbose: bool) -> str:
    """Object file of the Python entry points (host code)."""
    obj = os.path.join(BUILD_DIR, "mx_torch.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, "-isystem", os.path.join(torch, "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, "-c",
           os.path.join(CSRC, TORCH_SOURCE), "-o", obj]
    _run(cmd, verbose)
    return obj


def _run(cmd: list[str], verbose: bool = False) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{' '.join(cmd[-3:])} failed:\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        print(res.stdout + res.stderr, flush=True)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None,
          checked: bool = False) -> str:
    out_dir, lib = (CHECKED_DIR, CHECKED_LIB) if checked else (BUILD_DIR, LIB)
    torch = None if checked else _torch_dir()
    new_lib = force or _stale(lib)
    new_torch = torch is not None and (force or _stale(TORCH_LIB) or not fits_torch(torch))
    if not new_lib and not new_torch:
        return lib
    os.makedirs(out_dir, exist_ok=True)
    nvcc = _nvcc()
    flags = NVCC_FLAGS + (["-DMX_CHECKED=1"] if checked else []) + (extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(out_dir, os.path.splitext(src)[0] + ".o")
        _run([nvcc, *ARCH, *flags, "-c", os.path.join(CSRC, src), "-o", obj], verbose)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        torch_obj = ex.submit(_compile_torch, torch, verbose) if new_torch else None
        objs = list(ex.map(compile_one, SOURCES)) if new_lib else []
    if new_lib:
        tmp = lib + f".tmp{os.getpid()}"
        _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, lib)
    if torch_obj is not None:
        tmp = TORCH_LIB + f".tmp{os.getpid()}"
        _run(["g++", "-shared", "-o", tmp, torch_obj.result(), "-L", out_dir, "-l:libmx.so", "-Wl,-rpath,$ORIGIN",
              "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"])
        os.replace(tmp, TORCH_LIB)
        with open(TORCH_STAMP, "w") as f:
            f.write(_torch_stamp(torch))
    return lib


if __name__ == "__main__":
    print(build(force=True, verbose=True))
