"""The binding's short cut (csrc/torch_calls.cpp): when it is loaded and how it is built (no GPU)."""
import os
import subprocess
import sys

import pytest

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
