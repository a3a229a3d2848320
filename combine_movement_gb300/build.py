"""Build libep_gb300.so in-tree for sm_103a (nvcc, one -gencode, TUs compiled
in parallel, no cmake), and the binding's extension _calls (the C compiler).
``python -m combine_movement_gb300.build`` or ``build()``; skipped when they are
newer than every source. Without Python.h the library is built alone."""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import fcntl
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_objs")
LIB_PATH = os.path.join(PKG, "libep_gb300.so")
# (with the interpreter's tag: another interpreter neither finds it fresh nor loads it)
CALLS_PATH = os.path.join(PKG, "_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
CALLS_SOURCE = os.path.join(CSRC, "calls.c")

GENCODE = "arch=compute_103a,code=sm_103a"
NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo", f"-gencode={GENCODE}",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills",
]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libep_gb300.so")
    return cand


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(p) > t for p in _inputs())


@contextlib.contextmanager
def _alone(folder: str):
    """One build at a time in `folder` (ranks and test workers each ask for one); the
    ones that waited find it done."""
    os.makedirs(folder, exist_ok=True)
    with open(os.path.join(folder, ".lock"), "w") as f:
        fcntl.flock(f, fcntl.LOCK_EX)
        yield


def _untagged() -> str:
    """The extension without a tag, which any interpreter would load."""
    return os.path.join(os.path.dirname(CALLS_PATH), "_calls.so")


def calls_stale() -> bool:
    if os.path.exists(_untagged()) or not os.path.exists(CALLS_PATH):
        return True
    t = os.path.getmtime(CALLS_PATH)
    return any(os.path.getmtime(p) > t for p in (CALLS_SOURCE, os.path.join(INCLUDE, "ep.h")))


def build_calls(force: bool = False) -> str:
    """Build the binding's extension, where Python.h is there; returns its path."""
    if force or calls_stale():
        with _alone(OBJ_DIR):
            _build_calls(force)
    return CALLS_PATH


def _build_calls(force: bool) -> None:
    if not force and not calls_stale():
        return
    if os.path.exists(_untagged()):
        os.remove(_untagged())
    cc = shutil.which("gcc") or shutil.which("cc")
    headers = sysconfig.get_paths()["include"]
    missing = "a C compiler" if cc is None else "Python.h"
    if cc is None or not os.path.exists(os.path.join(headers, "Python.h")):
        warnings.warn(f"the binding's extension is not built: {missing} was not found (the router's "
                      "and the dense products' calls need it, the others do not)")
        return
    tmp = CALLS_PATH + ".tmp"
    cmd = [cc, "-O2", "-shared", "-fPIC", "-fvisibility=hidden", "-Wall", "-I", INCLUDE,
           "-I", headers, CALLS_SOURCE, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cc} failed on {CALLS_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS_PATH)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None,
          out_dir: str | None = None) -> str:
    """Build the library; returns its path. With ``out_dir`` the objects and
    the library go there instead of in-tree (used to build the measured
    alternatives, e.g. ``extra_flags=["-DEP_COMBINE_MODE=1"]``, beside the
    default library)."""
    lib_path = os.path.join(out_dir, "libep_gb300.so") if out_dir else LIB_PATH
    obj_dir = os.path.join(out_dir, "_objs") if out_dir else OBJ_DIR
    if out_dir is None and not force and not calls_stale() and not is_stale():
        return LIB_PATH  # (nothing is written where nothing is to be built)
    with _alone(obj_dir):
        if out_dir is not None or force or is_stale():
            _build_library(lib_path, obj_dir, verbose, extra_flags)
        if out_dir is None:
            _build_calls(force)
    return lib_path


def _build_library(lib_path: str, obj_dir: str, verbose: bool,
                   extra_flags: list[str] | None) -> None:
    nvcc = _nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(obj_dir, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, *flags, "-I", INCLUDE, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib_path + ".tmp"
    cmd = [nvcc, "-shared", f"-gencode={GENCODE}", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
