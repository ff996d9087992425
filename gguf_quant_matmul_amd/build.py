"""Build libkq.so for gfx950 in-tree: ``python -m gguf_quant_matmul_amd.build``.

Compiles every ``csrc/*.hip`` with hipcc (one process per file, in parallel)
and links them into ``gguf_quant_matmul_amd/libkq.so``; then the host module
``_kqcall.so`` (``csrc/kq_call.cpp``), which passes Python tensors to it.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libkq.so")
CALL = os.path.join(HERE, "_kqcall.so")
ARCH = os.environ.get("KQ_OFFLOAD_ARCH", "gfx950")

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

FLAGS = [
    "-O3",
    "-std=c++17",
    "-fPIC",
    f"--offload-arch={ARCH}",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    # no packed-fp32 instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *FLAGS, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(line for line in (res.stdout + res.stderr).splitlines() if "packed-fp32-ops" not in line)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{out}")
    if verbose and out.strip():
        print(out)
    return obj


def _stale(src: str) -> bool:
    """True if src's object is missing or older than src or any header of csrc/."""
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if not os.path.exists(obj):
        return True
    newest = max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in glob.glob(os.path.join(CSRC, "*.h"))])
    return os.path.getmtime(obj) < newest


def _call_module(verbose: bool, incremental: bool) -> None:
    """Compile csrc/kq_call.cpp (plain C++ against torch's headers) and link it to libkq.so beside it.

    The library is whole without it (kq.py then calls through ctypes), so a machine that cannot build it, for want of
    torch, a C++ compiler or Python's headers, gets a warning; a module of an earlier build does not stay behind."""
    src = os.path.join(CSRC, "kq_call.cpp")
    deps = [src, os.path.join(HERE, os.pardir, "include", "kq.h")]
    if incremental and os.path.exists(CALL) and os.path.getmtime(CALL) >= max(map(os.path.getmtime, deps)):
        return
    if os.path.exists(CALL):
        os.remove(CALL)
    try:
        import torch

        root = os.path.dirname(torch.__file__)
        inc = os.path.join(root, "include")
        cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DKQ_TORCH="{torch.__version__}"',
               "-I" + inc, "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
               "-I" + sysconfig.get_paths()["include"], src, "-o", CALL + ".tmp",
               "-L" + HERE, "-l:libkq.so", "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
               "-Wl,-rpath,$ORIGIN"]
        res = subprocess.run(cmd, capture_output=True, text=True)
    except (ImportError, OSError) as e:  # no torch, no compiler
        why = str(e)
    else:
        why = res.stdout + res.stderr if res.returncode != 0 else ""
    if why:
        warnings.warn(f"{os.path.basename(CALL)} is not built, calls of the cache operators will go through ctypes:\n{why}",
                      RuntimeWarning, stacklevel=2)
        return
    os.replace(CALL + ".tmp", CALL)
    if verbose:
        print(f"built {CALL}")


def build(verbose: bool = False, incremental: bool = False) -> str:
    """Compile every source and link libkq.so; with incremental=True only the
    sources whose object is older than the source or a header are compiled."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    todo = [s for s in srcs if _stale(s)] if incremental else srcs
    workers = max(1, min(len(todo), int(os.environ.get("MAX_JOBS", "8")), 16))
    with cf.ThreadPoolExecutor(max_workers=workers) as ex:
        list(ex.map(lambda s: _compile(s, verbose), todo))
    objs = [os.path.join(BUILD, os.path.basename(s) + ".o") for s in srcs]
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}{res.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    _call_module(verbose, incremental)
    return LIB


if __name__ == "__main__":
    build(verbose=True, incremental="--incremental" in sys.argv)
    sys.exit(0)
