"""The binding's short cut (csrc/torch_calls.cpp): when it is loaded and how it is built (no GPU)."""
import os
import shutil
import subprocess
import sys

import pytest

from kernelized_linear_attention_fwd_b200 import binding
from kernelized_linear_attention_fwd_b200.csrc import build as kbuild

ROOT = kbuild.ROOT


@pytest.fixture(scope="module", autouse=True)
def _built():
    kbuild.build()


def python(code):
    env = dict(os.environ, PYTHONPATH=ROOT)
    return subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_loading_the_library_does_not_load_torch():
    r = python("import sys\n"
               "import kernelized_linear_attention_fwd_b200 as K\n"
               "K.kata_version(), K.kata_cross_forward_workspace_bytes(1, 1, 1, 1, 100, 64, 1)\n"
               "assert 'torch' not in sys.modules")
    assert r.returncode == 0, r.stderr[-2000:]


def test_the_short_cut_is_found_by_the_first_call_with_tensors():
    r = python("import kernelized_linear_attention_fwd_b200 as K\n"
               "from kernelized_linear_attention_fwd_b200 import binding\n"
               "K.kata_version()\n"
               "import torch\n"
               "x = torch.zeros(1, 2, 3, 16)\n"
               "try: K.kata_cross_forward(x, x, x)\n"
               "except K.KataError: pass\n"
               "assert binding._calls is not None")
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build's outputs in an empty folder, and nvcc replaced by a copy of nothing."""
    monkeypatch.setattr(kbuild, "OUT", str(tmp_path / "libkata.so"))
    monkeypatch.setattr(kbuild, "PKG", str(tmp_path))
    ran = []

    def check_call(cmd):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(kbuild.subprocess, "check_call", check_call)
    return tmp_path, ran


def names(folder):
    return sorted(p.name for p in folder.iterdir())


def earlier(folder):
    """Short cuts of other Pythons and torches, older than their sources."""
    for name in ("_calls.so", "_calls-torch1.0.cpython-38-x86_64-linux-gnu.so", binding.calls_file()):
        (folder / name).write_text("")
        os.utime(folder / name, (1, 1))


def test_the_library_is_built_without_torch(elsewhere, monkeypatch):
    folder, ran = elsewhere
    earlier(folder)
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails
    assert kbuild.build(force=True) == str(folder / "libkata.so")
    assert len(ran) == 1 and names(folder) == ["libkata.so"]


@pytest.mark.parametrize("cmd", [["false"], ["/no/such/compiler"]])
def test_the_library_is_built_where_the_short_cut_fails(elsewhere, monkeypatch, cmd):
    folder, ran = elsewhere
    earlier(folder)
    (folder / binding.calls_file()).write_text("of a build just now")
    monkeypatch.setattr(kbuild, "calls_command", lambda out: cmd)
    kbuild.build(force=True)
    assert len(ran) == 1 and names(folder) == ["libkata.so"]


def test_another_process_removes_the_same_old_file(elsewhere, monkeypatch):
    folder, _ = elsewhere
    monkeypatch.setattr(kbuild.glob, "glob", lambda pattern: [str(folder / "_calls-gone.so")])
    monkeypatch.setattr(kbuild, "sources", lambda: [])
    monkeypatch.setattr(kbuild, "headers", lambda: [])
    monkeypatch.setattr(kbuild, "calls_command", lambda out: ["false"])
    kbuild.build(force=True)
    assert names(folder) == ["libkata.so"]


def test_a_failing_library_build_leaves_no_compiler_behind(elsewhere, monkeypatch):
    folder, _ = elsewhere
    monkeypatch.setattr(kbuild, "calls_command", lambda out: ["sh", "-c", "sleep 0.3; : > " + out])

    def fails(cmd):
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(kbuild.subprocess, "check_call", fails)
    with pytest.raises(subprocess.CalledProcessError):
        kbuild.build(force=True)
    assert names(folder) == [binding.calls_file()]  # waited for


def test_headers_are_those_of_the_toolkit_in_use(tmp_path, monkeypatch):
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "cuda_runtime_api.h").write_text("")
    (tmp_path / "bin").mkdir()
    nvcc = tmp_path / "bin" / "nvcc"
    nvcc.write_text("#!/bin/sh")
    nvcc.chmod(0o755)
    for name in ("CUDA_HOME", "CUDA_PATH"):
        monkeypatch.delenv(name, raising=False)
    monkeypatch.setenv("NVCC", str(nvcc))
    assert kbuild.cuda_include() == str(tmp_path / "include")
    monkeypatch.setenv("CUDA_HOME", "/no/such/place")
    assert kbuild.cuda_include() == str(tmp_path / "include")


def test_the_short_cut_of_another_torch_or_python_is_not_loaded(tmp_path, monkeypatch):
    import importlib.machinery

    import torch

    lib, mine = binding.load_library(), binding.calls_file()
    shutil.copy(os.path.join(kbuild.PKG, mine), tmp_path / mine)
    monkeypatch.setattr(binding, "_HERE", str(tmp_path))
    for where, name, value in ((torch, "__version__", torch.__version__ + ".1"),
                               (importlib.machinery, "EXTENSION_SUFFIXES", [".cpython-399-x86_64-linux-gnu.so"])):
        with monkeypatch.context() as m:
            m.setattr(binding, "_calls", None)
            m.setattr(where, name, value)
            binding._bind_calls(lib)
            assert binding._calls is None and binding.calls_file() != mine
            # nor under the name of a build that recorded nothing
            shutil.copy(tmp_path / mine, tmp_path / "_calls.so")
            binding._bind_calls(lib)
            assert binding._calls is None
    with monkeypatch.context() as m:
        m.setattr(binding, "_calls", None)
        binding._bind_calls(lib)
        assert binding._calls is not None
