"""Build libgtr.so in-tree with nvcc for sm_100a (B200), and, where torch is installed,
_gtr_torch.so, the argument marshalling of the state space calls for torch tensors, with g++.

Usage: ``python gated_token_recurrence_b200/build.py [--force] [--verbose] [--ptxas]``
(run as a script: importing the package itself needs the built library).
The library is written next to this file so that it travels with the source
tree; it is not installed anywhere.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libgtr.so")
TORCH_LIB = os.path.join(HERE, "_gtr_torch.so")
TORCH_SRC = os.path.join(CSRC, "gtr_torch.cpp")
OBJDIR = os.path.join(CSRC, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_binding_obstacle():
    """What keeps the marshalling module from being built here, or None."""
    import shutil
    import sysconfig
    try:
        import torch  # noqa: F401
    except ImportError:
        return "torch is not installed"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h is not installed"
    if shutil.which("g++") is None:
        return "g++ is not installed"
    return None


def torch_binding_target() -> str:
    """What the module is compiled for: it is loaded and kept for exactly this."""
    import sysconfig
    import torch
    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')}"


def build_torch_binding(force: bool = False, verbose: bool = False):
    """Compile csrc/gtr_torch.cpp against the installed torch's headers.  Where torch, the Python
    headers or g++ are missing it only says so: the C-ABI library does not need the module."""
    deps = [TORCH_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))
    stamp = os.path.join(OBJDIR, "_gtr_torch.target")  # what the module beside it was compiled for
    fresh = os.path.exists(TORCH_LIB) and all(os.path.getmtime(d) <= os.path.getmtime(TORCH_LIB) for d in deps)
    obstacle = _torch_binding_obstacle()
    if obstacle is not None:
        if (force or not fresh) and os.path.exists(TORCH_LIB):
            os.remove(TORCH_LIB)  # made for another gtr.h
        print(f"_gtr_torch.so not built: {obstacle}; the state space and block norm calls of the Python "
              "binding need it", file=sys.stderr)
        return None
    target = torch_binding_target()
    if not force and fresh and os.path.exists(stamp) and open(stamp).read() == target:
        return TORCH_LIB
    import sysconfig
    import torch
    root = os.path.dirname(torch.__file__)
    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DGTR_BUILT_FOR="{target}"', "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"), TORCH_SRC, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    done = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if done.returncode != 0:
        raise RuntimeError("g++ failed:\n" + done.stdout.decode(errors="replace"))
    os.replace(tmp, TORCH_LIB)
    os.makedirs(OBJDIR, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(target)
    return TORCH_LIB


def build(force: bool = False, verbose: bool = False, ptxas_report: bool = False) -> str:
    """Compile every csrc/*.cu into libgtr.so (objects in csrc/_build, linked with cudart static),
    then the binding's module where torch is installed."""
    if force or _stale():
        _build_library(verbose, ptxas_report)
    build_torch_binding(force, verbose)
    return LIB


def _build_library(verbose: bool, ptxas_report: bool) -> None:
    os.makedirs(OBJDIR, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if ptxas_report:
            cmd += ["-Xptxas", "-v"]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    failed = []
    for src, pr in procs:
        out, _ = pr.communicate()
        text = out.decode(errors="replace")
        if pr.returncode != 0:
            failed.append((src, text))
        elif verbose or ptxas_report:
            print(text, end="")
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError("nvcc failed:\n" + msg)
    tmp = LIB + f".tmp{os.getpid()}"
    link = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs,
            "-Xcompiler", "-fPIC"]
    if verbose:
        print(" ".join(link), flush=True)
    subprocess.run(link, check=True)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv,
          ptxas_report="--ptxas" in sys.argv)
    print(LIB)
