"""Builds libkata.so (the C-ABI library) for sm_100a with nvcc.

    python kernelized_linear_attention_fwd_b200/csrc/build.py [--verbose]

The shared object lands in the package directory beside the Python binding.
Beside it lands _calls.so, the binding's short cut (torch_calls.cpp, g++ against
torch's headers); without those headers it is left out and the binding works
without it.  Cross-compiles without a GPU.  `--verbose` adds -Xptxas -v (registers, spills,
shared memory per kernel).
"""
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(HERE)
ROOT = os.path.dirname(PKG)
OUT = os.path.join(PKG, "libkata.so")

CALLS_SRC = os.path.join(HERE, "torch_calls.cpp")
CALLS_OUT = os.path.join(PKG, "_calls.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
    "-I", os.path.join(ROOT, "include"),
]


def sources():
    return sorted(glob.glob(os.path.join(HERE, "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(HERE, "*.cuh"))) + [os.path.join(ROOT, "include", "kata.h")]


def up_to_date():
    if not os.path.exists(OUT):
        return False
    t = os.path.getmtime(OUT)
    return all(os.path.getmtime(f) <= t for f in sources() + headers() + [__file__])


def calls_command(out):
    """The g++ command of _calls.so, or None where a header it needs is missing."""
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], "/usr/local/cuda/include"]
    needed = [os.path.join(inc, "ATen", "ATen.h"), os.path.join(dirs[2], "Python.h"),
              os.path.join(dirs[3], "cuda_runtime_api.h")]
    if not all(os.path.exists(f) for f in needed):
        return None
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w", CALLS_SRC, "-o", out]
            + ["-I" + d for d in dirs]
            + ["-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + lib])


def build_calls(force=False):
    """Starts building _calls.so if it is missing or older than its sources; returns a
    function that waits for it."""
    deps = [CALLS_SRC, os.path.join(ROOT, "include", "kata.h"), __file__]
    if (not force and os.path.exists(CALLS_OUT)
            and all(os.path.getmtime(f) <= os.path.getmtime(CALLS_OUT) for f in deps)):
        return lambda: None
    tmp = CALLS_OUT + ".tmp%d" % os.getpid()
    cmd = calls_command(tmp)
    if cmd is None:
        print("torch or Python headers not found: built without _calls.so")
        return lambda: None
    proc = subprocess.Popen(cmd)

    def finish():
        if proc.wait() != 0:
            raise subprocess.CalledProcessError(proc.returncode, cmd)
        os.replace(tmp, CALLS_OUT)

    return finish


def build(force=False, verbose=False):
    finish = build_calls(force)
    if force or verbose or not up_to_date():
        nvcc = os.environ.get("NVCC", "nvcc")
        tmp = OUT + ".tmp%d" % os.getpid()
        cmd = [nvcc] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + sources() + ["-o", tmp]
        subprocess.check_call(cmd)
        os.replace(tmp, OUT)
    finish()
    return OUT


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
