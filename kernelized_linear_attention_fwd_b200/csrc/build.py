"""Builds libkata.so (the C-ABI library) for sm_100a with nvcc.

    python kernelized_linear_attention_fwd_b200/csrc/build.py [--verbose]

The shared object lands in the package directory beside the Python binding.
Beside it lands _calls-torch<version>.<Python's suffix>.so, the binding's short cut
(torch_calls.cpp, g++ against torch's headers); where torch, a header or the compiler is
missing, or the compiler fails, it is left out and the binding works without it.
Cross-compiles without a GPU.  `--verbose` adds -Xptxas -v (registers, spills, shared
memory per kernel).
"""
import contextlib
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(HERE)
ROOT = os.path.dirname(PKG)
OUT = os.path.join(PKG, "libkata.so")

CALLS_SRC = os.path.join(HERE, "torch_calls.cpp")

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


def cuda_include():
    """The CUDA toolkit's headers: of CUDA_HOME, of the compiler in use, or in the usual place."""
    nvcc = shutil.which(os.environ.get("NVCC", "nvcc"))
    homes = [os.environ.get("CUDA_HOME"), os.environ.get("CUDA_PATH"),
             nvcc and os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "/usr/local/cuda"]
    found = [d for d in (os.path.join(h, "include") for h in homes if h)
             if os.path.exists(os.path.join(d, "cuda_runtime_api.h"))]
    return found[0] if found else None


def calls_out():
    """Where the short cut for the running Python and torch lies, or None without torch."""
    try:
        import torch  # noqa: F401
    except ImportError:
        return None
    spec = importlib.util.spec_from_file_location("binding", os.path.join(HERE, "..", "binding.py"))
    binding = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(binding)
    return os.path.join(PKG, binding.calls_file())


def calls_command(out):
    """The g++ command of the short cut, or None where a header it needs is missing."""
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    python, cuda = sysconfig.get_paths()["include"], cuda_include()
    needed = [os.path.join(inc, "ATen", "ATen.h"), os.path.join(python, "Python.h")]
    if cuda is None or not all(os.path.exists(f) for f in needed):
        return None
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), python, cuda]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w", CALLS_SRC, "-o", out]
            + ["-I" + d for d in dirs]
            + ["-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + lib])


def build_calls(force=False):
    """Starts building the short cut if it is missing or older than its sources; returns a
    function that waits for it.  Where it cannot be built it is left out.  Older ones, which were
    built for other declarations, are removed, whatever torch and Python they are for."""
    deps = [CALLS_SRC, os.path.join(ROOT, "include", "kata.h"), __file__]
    for f in glob.glob(os.path.join(PKG, "_calls*.so")):
        with contextlib.suppress(FileNotFoundError):  # another process builds too
            if any(os.path.getmtime(d) > os.path.getmtime(f) for d in deps):
                os.remove(f)
    out = calls_out()
    if out and os.path.exists(out) and not force:
        return lambda: None

    def without(why):
        print(why + ": built without " + os.path.basename(out or "_calls.so"))
        if out:
            with contextlib.suppress(FileNotFoundError):
                os.remove(out)

    tmp = "%s.tmp%d" % (out, os.getpid())
    cmd = calls_command(tmp) if out else None
    if cmd is None:
        return lambda: without("torch or headers not found")
    try:
        proc = subprocess.Popen(cmd)
    except OSError:
        return lambda: without(cmd[0] + " not found")

    def finish():
        if proc.wait() == 0:
            os.replace(tmp, out)
        else:
            without("%s failed (%d)" % (cmd[0], proc.returncode))

    return finish


def build(force=False, verbose=False):
    finish = build_calls(force)
    try:
        if force or verbose or not up_to_date():
            nvcc = os.environ.get("NVCC", "nvcc")
            tmp = OUT + ".tmp%d" % os.getpid()
            cmd = [nvcc] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + sources() + ["-o", tmp]
            subprocess.check_call(cmd)
            os.replace(tmp, OUT)
    finally:
        finish()
    return OUT


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
