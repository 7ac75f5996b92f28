"""Build libspecverify.so in place with nvcc for sm_103a.

    python -m speculative_decoding_verification_31_gb300.build
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libspecverify.so")
CHECKED_LIB = os.path.join(PKG, "libspecverify_checked.so")  # SPECVERIFY_CHECKED: index checks
SOURCES = ["specverify.cu", "operators.cu"]
DEPS = SOURCES + ["kernels.cuh", "vocab.cuh", "device_common.cuh", "philox.cuh", "lmhead.cuh", "tensor_core.cuh",
                  "probs.cuh", "norm.cuh", "linear.cuh", "internal.h"]
BINDING_DEPS = ["binding.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def cuda_home() -> str:
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if home and os.path.exists(os.path.join(home, "bin", "nvcc")):
        return home
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def nvcc_command(out: str = LIB, extra=()) -> list:
    home = cuda_home()
    return [os.path.join(home, "bin", "nvcc"), *ARCH, "-O3", "-std=c++17", "-lineinfo",
            "--shared", "--threads", "0", "-Xcompiler", "-fPIC", "-cudart", "shared",
            f"-I{INCLUDE}", f"-I{CSRC}", "-Xlinker", f"-rpath={os.path.join(home, 'lib64')}",
            *extra, "-o", out, *[os.path.join(CSRC, s) for s in SOURCES]]


def binding_path() -> str:
    """The compiled argument marshalling (a Python extension) for the running interpreter and PyTorch,
    whose versions are in its name: after a change of either it is built again."""
    import sysconfig

    import torch
    tag = "".join(c if c.isalnum() else "_" for c in torch.__version__)
    return os.path.join(PKG, f"_binding.torch_{tag}{sysconfig.get_config_var('EXT_SUFFIX')}")


def binding_command() -> list:
    """g++ on the Python extension, against the running interpreter's headers and torch's."""
    import sysconfig

    import torch
    t = torch.__path__[0]
    inc = [sysconfig.get_paths()["include"], os.path.join(t, "include"),
           os.path.join(t, "include", "torch", "csrc", "api", "include"), os.path.join(cuda_home(), "include"), INCLUDE]
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", *(f"-I{i}" for i in inc),
            os.path.join(CSRC, "binding.cpp"), "-o", binding_path(), f"-L{os.path.join(t, 'lib')}",
            f"-Wl,-rpath,{os.path.join(t, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def up_to_date(out: str = LIB, sources=DEPS) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    deps = [os.path.join(CSRC, d) for d in sources] + [os.path.join(INCLUDE, "specverify.h")]
    return all(os.path.getmtime(d) <= t for d in deps)


def start(cmd: list, verbose: bool):
    if verbose:
        print(" ".join(cmd))
    return cmd, subprocess.Popen(cmd)


def build(force: bool = False, verbose: bool = False, extra=(), checked: bool = True) -> str:
    """Compile libspecverify.so, its index-checked variant libspecverify_checked.so (unless
    checked=False) and the Python extension, side by side.  Returns the library's path.  The extension
    also needs Python's and PyTorch's headers; where it cannot be built the library still is, for C
    callers and the calls that go through ctypes, and a warning says so (the calls that need it raise)."""
    jobs = []
    if force or not up_to_date(LIB):
        jobs.append(start(nvcc_command(out=LIB, extra=list(extra)), verbose))
    if checked and (force or not up_to_date(CHECKED_LIB)):
        jobs.append(start(nvcc_command(out=CHECKED_LIB, extra=["-DSPECVERIFY_CHECKED", *extra]), verbose))
    missing = None
    try:
        if force or not up_to_date(binding_path(), BINDING_DEPS):
            if os.path.exists(binding_path()):
                os.remove(binding_path())  # (where the build fails, an old one is not called)
            cmd, pr = start(binding_command(), verbose)
            if pr.wait() != 0:
                missing = f"{cmd[0]} exited with {pr.returncode}"
    except (ImportError, OSError) as e:  # no PyTorch, no compiler
        missing = str(e)
    failed = [cmd for cmd, pr in jobs if pr.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    if missing:
        print(f"warning: the Python extension was not built ({missing}); spec_verify_probs, spec_rms_norm, "
              "spec_rms_norm_fp8 and spec_linear can be called from C but not from Python", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
