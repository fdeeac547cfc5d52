"""Build libgdr.so (the HIP kernels and the C ABI) for gfx950 with hipcc, and
the binding's CPython extension _marshal.so with the host compiler.

``python -m gated_delta_rule_40_amd.build`` or ``build_library()`` compiles
every source under ``csrc/`` to an object in ``_build/`` (in parallel) and
links them into ``gated_delta_rule_40_amd/libgdr.so``; ``csrc/python/`` goes
into ``gated_delta_rule_40_amd/_marshal.so``.  It always recompiles.  The C
library needs hipcc alone; without torch or Python's headers the extension, which
only the binding uses, is left out.
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
BUILD_DIR = ROOT / "_build"
LIB_PATH = PKG / "libgdr.so"
MARSHAL_PATH = PKG / "_marshal.so"
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-function",
    "-ffp-contract=fast",
    # Packed fp32 arithmetic stays off: plain scalar fp32 code only.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{ROOT / 'include'}",
    f"-I{CSRC}",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libgdr.so)")


def sources() -> list[Path]:
    return sorted(CSRC.glob("*.hip")) + sorted(CSRC.glob("*.cpp"))


def _compile(src: Path, verbose: bool) -> Path:
    obj = BUILD_DIR / (src.name + ".o")
    cmd = [hipcc(), *HIPCC_FLAGS, "-c", str(src), "-o", str(obj)]
    if src.suffix == ".cpp":
        cmd.insert(1, "-x")
        cmd.insert(2, "hip")
    res = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the packed-fp32 target feature and says so.
    noise = "is not a recognized feature for this target"
    msgs = [ln for ln in (res.stdout + res.stderr).splitlines() if noise not in ln]
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src.name}:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs), file=sys.stderr)
    return obj


def _lacking() -> str | None:
    """What the binding's extension would need and is not there."""
    if importlib.util.find_spec("torch") is None:
        return "torch"
    if not (Path(sysconfig.get_paths()["include"]) / "Python.h").exists():
        return "Python.h"
    return None


def _build_marshal() -> None:
    lacking = _lacking()
    if lacking:
        print(f"{MARSHAL_PATH.name} is not built: no {lacking}", file=sys.stderr)
        return
    import torch

    t = Path(torch.__file__).resolve().parent
    tmp = MARSHAL_PATH.with_name(f"{MARSHAL_PATH.name}.tmp{os.getpid()}")
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", str(t / "include"),
           "-isystem", str(t / "include" / "torch" / "csrc" / "api" / "include"),
           "-isystem", sysconfig.get_paths()["include"], str(CSRC / "python" / "marshal.cpp"),
           f"-L{t / 'lib'}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", str(tmp)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("compiling _marshal.so failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, MARSHAL_PATH)


def build_library(verbose: bool = False, jobs: int | None = None) -> Path:
    BUILD_DIR.mkdir(exist_ok=True)
    srcs = sources()
    jobs = jobs or min(len(srcs), max(1, (os.cpu_count() or 2)), 16)
    with ThreadPoolExecutor(jobs) as ex:
        marshal = ex.submit(_build_marshal)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = LIB_PATH.with_name(f"{LIB_PATH.name}.tmp{os.getpid()}")
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *map(str, objs), "-o", str(tmp)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, LIB_PATH)
    marshal.result()  # raises if it failed, with the library in place
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(verbose=True))
