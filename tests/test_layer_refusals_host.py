"""Every refusal of the head norm's and cross attention's entry points beside a call that is
accepted, on the argument checks alone (tests/csrc/layer_abi_stub.cu: launches succeed, no
GPU): the tables of tests/test_layer_abi_host.py, whose addresses the library itself
refuses last of all, so that there a lost check goes unseen."""
import ctypes
import os
import subprocess

import pytest

from kernelized_linear_attention_fwd_b200 import binding as E
from kernelized_linear_attention_fwd_b200.csrc import build as kbuild
from tests import test_layer_abi_host as A
from tests.test_layer_abi_host import INV, UNS, WS, at

OK = E.KATA_OK
SRC = os.path.join(kbuild.ROOT, "tests", "csrc", "layer_abi_stub.cu")


@pytest.fixture(scope="module")
def stub(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("stub") / "libstub.so")
    subprocess.check_call([os.environ.get("NVCC", "nvcc"), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17",
                           "--expt-relaxed-constexpr", "-I", os.path.join(kbuild.ROOT, "include"), "-Xcompiler",
                           "-fPIC", "-shared", SRC, "-o", out])
    real, lib = E.load_library(), ctypes.CDLL(out)
    for name in E.EXPORTS:
        if name.startswith(("kata_qk", "kata_cross")):
            getattr(lib, name).argtypes = getattr(real, name).argtypes
            getattr(lib, name).restype = getattr(real, name).restype
    lib.stub_foreign.argtypes = [ctypes.c_void_p]
    return lib


def cross_f(lib, **o):
    return A.cross(lib, "f", **o)


def cross_b(lib, **o):
    return A.cross(lib, "b", **o)


def table(test):
    """The rows of a parametrised test: (overrides, status)."""
    return next(m.args[1] for m in test.pytestmark if m.args[0] == "bad,status")


ROWS = ([(A.norm, r) for r in table(A.test_norm_refusals)]
        + [(A.norm_bwd, r) for r in table(A.test_norm_backward_refusals)]
        + [(f, r) for f in (cross_f, cross_b) for r in table(A.test_cross_refusals)]
        + [(cross_f, r) for r in table(A.test_cross_forward_refusals)]
        + [(cross_b, r) for r in table(A.test_cross_backward_refusals)]
        # a gradient of one row that reaches a given tensor's memory
        + [(A.norm_bwd, (b, INV)) for b in (
            dict(dq=at(1)), dict(dk=at(0)), dict(dk=at(2)), dict(dq=at(3)), dict(dq=at(4)), dict(dq=at(5)),
            dict(dq=at(6)), dict(dq=at(7)), dict(dqw=at(0)), dict(dqw=at(2)), dict(dkw=at(3)), dict(dkw=at(5)),
            dict(dkw=at(9)), dict(dqw=at(9)), dict(dqw=at(6)), dict(dqw=at(7)), dict(gq=at(0, 8)), dict(gk=at(1, 8)),
            dict(dq=at(8, 8)), dict(dk=at(9, 2)), dict(dqw=at(10, 4)), dict(dkw=at(11, 8)), dict(dqs=None),
            dict(dks=None), dict(qs=None), dict(ks=None), dict(n=33), dict(eps=0.0), dict(ps=-1),
            dict(dqs=(1536, 516, 64)), dict(dqs=(1536, 512, -64)), dict(q=at(2, 2)), dict(k=at(3, 2)))]
        + [(A.norm_bwd, (dict(n=30), UNS)), (A.norm_bwd, (dict(d=48), UNS)), (A.norm_bwd, (dict(dt=2), UNS))]
        + [(A.norm, (b, INV)) for b in (
            dict(ko=at(0)), dict(ko=at(1)), dict(qo=at(1)), dict(qo=at(4)), dict(ko=at(5)), dict(ko=at(6)),
            dict(ko=at(7)), dict(qo=at(2, 8)), dict(ko=at(3, 8)), dict(k=at(1, 8)), dict(kw=at(5, 4)),
            dict(inv=at(6, 4)), dict(ks=(1536, 512, 68)), dict(ks=(-1536, 512, 64)), dict(ps=2 ** 41),
            dict(q=at(14), qs=(2 ** 46, 512, 64)))]
        + [(cross_f, (b, INV)) for b in (
            dict(k=at(2, 8)), dict(den=at(5, 4)), dict(out=at(7, 8)), dict(out=at(2)), dict(y=at(1)), dict(y=at(2)),
            dict(y=at(3)), dict(y=at(6)), dict(den=at(7)), dict(den=at(1)), dict(den=at(3)), dict(den=at(6)))]
        + [(cross_b, (b, INV)) for b in (
            dict(g=at(0, 8)), dict(k=at(2, 8)), dict(den=at(5, 8)), dict(dk=at(8, 8)), dict(dv=at(9, 8)),
            dict(out=at(0)), dict(out=at(4)), dict(out=at(5)), dict(dk=at(0)), dict(dk=at(1)), dict(dk=at(3)),
            dict(dk=at(4)), dict(dk=at(5)), dict(dk=at(6)), dict(dk=at(7)), dict(dv=at(1)), dict(dv=at(2)),
            dict(dv=at(3)), dict(dv=at(5)), dict(dv=at(6)))])


@pytest.mark.parametrize("call", [A.norm, A.norm_bwd, cross_f, cross_b], ids=lambda f: f.__name__)
def test_the_call_that_the_tables_vary_is_accepted(stub, call):
    n = stub.stub_launches()
    assert call(stub) == OK and stub.stub_launches() == n + 1


@pytest.mark.parametrize("row", range(len(ROWS)))
def test_refusals(stub, row):
    call, (bad, status) = ROWS[row]
    n = stub.stub_launches()
    assert call(stub, **bad) == status, (call.__name__, bad)
    assert stub.stub_launches() == n


@pytest.mark.parametrize("call,good", [
    (A.norm, dict(n=30, inter=1)), (A.norm, dict(pos=0)), (A.norm, dict(n=0, inv=0)), (A.norm, dict(qw=0, kw=0)),
    (A.norm, dict(k=0, ko=0, Hk=0, ks=None)), (A.norm, dict(qs=(0, 0, 0))), (A.norm, dict(T=1, qs=(512, 3, 64))),
    (A.norm, dict(dt=0, qs=(1536, 516, 64))), (A.norm, dict(ps=0)), (A.norm, dict(pos=at(7, 8))),
    (A.norm_bwd, dict(dqw=0, dkw=0)), (A.norm_bwd, dict(dk=at(8, 4 * 128))), (A.norm_bwd, dict(pos=0)),
    (A.norm_bwd, dict(k=0, gk=0, dk=0, dkw=0, Hk=0, ks=None, dks=None)),
    (cross_f, dict(y=0, den=0, n=0)), (cross_f, dict(n=at(6, 4))), (cross_b, dict(n=0)), (cross_b, dict(dt=0)),
    (cross_f, dict(Tq=1, H=2, Tk=100, Hkv=2, ws=0))])
def test_accepted(stub, call, good):
    assert call(stub, **good) == OK


@pytest.mark.parametrize("call,args", [
    (A.norm, [0, 1, 2, 3, 4, 5, 6, 7]), (A.norm_bwd, range(13)), (cross_f, [1, 2, 3, 4, 5, 6, 7, 10]),
    (cross_b, range(11))])
def test_every_address_is_checked_for_the_device(stub, call, args):
    try:
        for i in args:
            stub.stub_foreign(at(i))
            n = stub.stub_launches()
            # the forward's workspace only where it needs one
            size = dict(Tq=1, H=2, Tk=100000) if call is cross_f else {}
            assert call(stub, **size) == INV and stub.stub_launches() == n, i
    finally:
        stub.stub_foreign(None)


@pytest.mark.parametrize("call,size", [(A.norm_bwd, {}), (cross_f, dict(Tq=1, H=2, Tk=100000)), (cross_b, {})])
def test_workspaces(stub, call, size):
    if call is A.norm_bwd:
        need = stub.kata_qk_norm_rotate_backward_workspace_bytes(2, 3, 4, 2, 64)
    else:
        a = dict(B=2, H=4, Hkv=2, Tq=70, Tk=90, d=64, dt=1)
        a.update(size)
        q = stub.kata_cross_forward_workspace_bytes if call is cross_f else stub.kata_cross_backward_workspace_bytes
        need = q(*a.values())
    i = 12 if call is A.norm_bwd else 10
    assert need > 0 and call(stub, **size, wsb=need) == OK
    for bad in (dict(wsb=need - 1), dict(ws=0), dict(ws=at(i, 128)), dict(wsb=0)):
        assert call(stub, **{**size, "wsb": need, **bad}) == WS
