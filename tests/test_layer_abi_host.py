"""Host-side checks of the head norm's and cross attention's entry points (no GPU, no
kernel launched): every call here is one that the library must refuse, and the
workspace queries.  Like tests/test_abi_host.py it passes fake device addresses,
so it runs only where no GPU is visible."""
import ctypes

import pytest

from kernelized_linear_attention_fwd_b200 import binding as E
from kernelized_linear_attention_fwd_b200.csrc import build as kbuild

INV, UNS, WS = E.KATA_ERR_INVALID_ARG, E.KATA_ERR_UNSUPPORTED, E.KATA_ERR_WORKSPACE
F = 0x7F0000000000
STEP = 0x1000000000


@pytest.fixture(scope="module")
def lib():
    import torch

    if torch.cuda.is_available():
        pytest.skip("host-side ABI checks use fake device pointers: run without a GPU")
    kbuild.build()
    return E.load_library()


def at(i, off=0):
    return F + i * STEP + off


def vp(x):
    return ctypes.c_void_p(x) if x else None


def st3(*s):
    return (ctypes.c_int64 * 3)(*s)


def norm(lib, **o):
    a = dict(q=at(0), k=at(1), qo=at(2), ko=at(3), qw=at(4), kw=at(5), inv=at(6), pos=at(7), B=2, T=3, Hq=4, Hk=2,
             d=64, n=32, qs=(3 * 512, 512, 64), ks=(3 * 512, 512, 64), ps=3, eps=1e-6, inter=0, dt=1)
    a.update(o)
    return lib.kata_qk_norm_rotate(vp(a["q"]), vp(a["k"]), vp(a["qo"]), vp(a["ko"]), vp(a["qw"]), vp(a["kw"]),
                                   vp(a["inv"]), vp(a["pos"]), a["B"], a["T"], a["Hq"], a["Hk"], a["d"], a["n"],
                                   st3(*a["qs"]) if a["qs"] else None, st3(*a["ks"]) if a["ks"] else None, a["ps"],
                                   a["eps"], a["inter"], a["dt"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=0), INV), (dict(qo=0), INV), (dict(ko=0), INV), (dict(k=0), INV), (dict(Hk=0), INV),
    (dict(q=at(0, 2)), INV), (dict(qw=at(4, 4)), INV), (dict(pos=at(7, 4)), INV), (dict(inv=0), INV),
    (dict(B=0), INV), (dict(T=0), INV), (dict(Hq=0), INV), (dict(Hk=-1), INV), (dict(d=0), INV),
    (dict(d=48), UNS), (dict(d=128), UNS), (dict(dt=2), UNS), (dict(n=33), INV), (dict(n=-1), INV),
    (dict(n=30), UNS), (dict(eps=0.0), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(qs=None), INV), (dict(ks=None), INV), (dict(qs=(3 * 512, 512, -64)), INV),
    (dict(qs=(3 * 512, 512, 68)), INV), (dict(qs=(3 * 512, 516, 64)), INV), (dict(qs=(2 ** 60, 512, 64)), INV),
    (dict(ps=-1), INV), (dict(qo=at(0)), INV), (dict(ko=at(2)), INV), (dict(qo=at(6)), INV), (dict(qo=at(7)), INV),
    (dict(B=2 ** 30, T=2 ** 30, qs=(0, 512, 64), ks=(0, 512, 64)), UNS),
])
def test_norm_refusals(lib, bad, status):
    assert norm(lib, **bad) == status


def test_norm_takes_every_number_of_neighbouring_pairs(lib):
    # 30 pairs are refused half-split only: interleaved they reach the device check
    assert norm(lib, n=30, inter=1) == INV
    assert norm(lib, n=30, inter=0) == UNS


def norm_bwd(lib, **o):
    need = lib.kata_qk_norm_rotate_backward_workspace_bytes(2, 3, 4, 2, 64)
    a = dict(gq=at(0), gk=at(1), q=at(2), k=at(3), qw=at(4), kw=at(5), inv=at(6), pos=at(7), dq=at(8), dk=at(9),
             dqw=at(10), dkw=at(11), B=2, T=3, Hq=4, Hk=2, d=64, n=32, qs=(1536, 512, 64), ks=(1536, 512, 64),
             dqs=(1536, 512, 64), dks=(1536, 512, 64), ps=3, eps=1e-6, inter=0, dt=1, ws=at(12), wsb=need)
    a.update(o)
    s = {x: st3(*a[x]) if a[x] else None for x in ("qs", "ks", "dqs", "dks")}
    return lib.kata_qk_norm_rotate_backward(
        *[vp(a[x]) for x in ("gq", "gk", "q", "k", "qw", "kw", "inv", "pos", "dq", "dk", "dqw", "dkw")], a["B"],
        a["T"], a["Hq"], a["Hk"], a["d"], a["n"], s["qs"], s["ks"], s["dqs"], s["dks"], a["ps"], a["eps"],
        a["inter"], a["dt"], vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(gq=0), INV), (dict(gk=0), INV), (dict(dq=0), INV), (dict(dk=0), INV),
    (dict(k=0, Hk=0), INV),                              # gradients of keys that are not there
    (dict(dqs=(1536, 512, 32)), INV), (dict(dqs=(512, 512, 64)), INV), (dict(dqs=(1536, 0, 64)), INV),
    (dict(dq=at(2)), INV), (dict(dq=at(0)), INV), (dict(dk=at(3)), INV),
    (dict(dk=at(8)), INV),                               # the same rows twice
    (dict(dk=at(8, 3 * 128)), INV),                      # heads of dk over those of dq
    (dict(dk=at(8, 7 * 128)), INV),                      # dk's last head reaches dq's next token
    (dict(dqw=at(8)), INV), (dict(dkw=at(10)), INV), (dict(dqw=at(4)), INV),
    (dict(ws=0), WS), (dict(wsb=16), WS), (dict(ws=at(12, 16)), WS),
])
def test_norm_backward_refusals(lib, bad, status):
    assert norm_bwd(lib, **bad) == status


def test_norm_backward_takes_slices_of_one_buffer(lib):
    # past every host check: what is left is the address check of the fake pointers
    assert norm_bwd(lib, dk=at(8, 4 * 128), ws=0) == WS
    assert norm_bwd(lib, dk=at(8, 4 * 128)) == INV


def test_norm_workspace(lib):
    W = lib.kata_qk_norm_rotate_backward_workspace_bytes
    assert W(0, 1, 1, 1, 64) == 0 and W(1, 1, 1, 1, 48) == 0
    assert W(1, 1, 1, 0, 64) >= 2 * 64 * 4
    assert W(64, 4096, 16, 16, 64) <= 1 << 20  # bounded by the grid


def cross(lib, fn, **o):
    a = dict(g=at(0), q=at(1), k=at(2), v=at(3), y=at(4), den=at(5), n=at(6), out=at(7), dk=at(8), dv=at(9), B=2,
             H=4, Hkv=2, Tq=70, Tk=90, d=64, dt=1, ws=at(10), wsb=1 << 30)
    a.update(o)
    size = [a[x] for x in ("B", "H", "Hkv", "Tq", "Tk", "d", "dt")]
    if fn == "f":
        return lib.kata_cross_forward(vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["n"]), vp(a["out"]), *size,
                                      vp(a["y"]), vp(a["den"]), vp(a["ws"]), a["wsb"], None)
    return lib.kata_cross_backward(vp(a["g"]), vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["y"]), vp(a["den"]),
                                   vp(a["n"]), vp(a["out"]), vp(a["dk"]), vp(a["dv"]), *size, vp(a["ws"]),
                                   a["wsb"], None)


SIZES = [(dict(B=0), INV), (dict(H=0), INV), (dict(Hkv=0), INV), (dict(Hkv=3), INV), (dict(Tq=0), INV),
         (dict(Tk=0), INV), (dict(Tk=-4), INV), (dict(d=48), UNS), (dict(d=128), UNS), (dict(dt=3), UNS),
         (dict(Tq=2 ** 31 - 1), UNS), (dict(H=2 ** 10, Hkv=1, Tq=2 ** 22), UNS), (dict(Tk=2 ** 31 - 100), UNS),
         (dict(B=2 ** 20, H=2 ** 10, Hkv=2 ** 10, Tq=2 ** 12), UNS)]


@pytest.mark.parametrize("fn", ["f", "b"])
@pytest.mark.parametrize("bad,status", SIZES + [
    (dict(q=0), INV), (dict(k=0), INV), (dict(v=0), INV), (dict(out=0), INV), (dict(q=at(1, 8)), INV),
    (dict(v=at(3, 2)), INV), (dict(y=at(4, 4)), INV), (dict(n=at(6, 2)), INV), (dict(out=at(1)), INV),
    (dict(out=at(3)), INV), (dict(out=at(6)), INV), (dict(out=at(1, 128)), INV)])
def test_cross_refusals(lib, fn, bad, status):
    assert cross(lib, fn, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(y=at(7)), INV), (dict(den=at(4)), INV), (dict(den=at(2)), INV),
    (dict(Tq=1, H=2, Tk=100000, ws=0), WS), (dict(Tq=1, H=2, Tk=100000, wsb=128), WS),
    (dict(Tq=1, H=2, Tk=100000, ws=at(10, 64)), WS)])
def test_cross_forward_refusals(lib, bad, status):
    assert cross(lib, "f", **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(g=0), INV), (dict(y=0), INV), (dict(den=0), INV), (dict(dk=0), INV), (dict(dv=0), INV),
    (dict(dk=at(9)), INV), (dict(dv=at(7)), INV), (dict(dk=at(2)), INV), (dict(dv=at(0)), INV),
    (dict(dv=at(4)), INV), (dict(ws=0), WS), (dict(wsb=255), WS), (dict(ws=at(10, 128)), WS)])
def test_cross_backward_refusals(lib, bad, status):
    assert cross(lib, "b", **bad) == status


def test_norm_workspace_limits(lib):
    W = lib.kata_qk_norm_rotate_backward_workspace_bytes
    top = 2 ** 31 - 2 ** 17
    assert W(1, top - 1, 1, 1, 64) > 0 and W(top - 1, 1, 1, 1, 64) > 0
    assert W(1, top, 1, 1, 64) == 0 and W(top, 1, 1, 1, 64) == 0
    assert W(1, 2 ** 31 - 1, 1, 1, 64) == 0 and W(2 ** 31 - 1, 1, 1, 1, 64) == 0
    # a row of partial sums per block, which a single token has few of
    assert 0 < W(1, 1, 1, 1, 64) <= 2 * 64 * 4 + 255 and W(1, 10 ** 6, 32, 32, 16) <= 4 * 148 * 2 * 16 * 4 + 255


def test_cross_workspace(lib):
    W, V = lib.kata_cross_forward_workspace_bytes, lib.kata_cross_backward_workspace_bytes
    for bad, _ in SIZES:
        a = dict(B=2, H=4, Hkv=2, Tq=70, Tk=90, d=64, dt=1)
        a.update(bad)
        assert W(*a.values()) == 0 and V(*a.values()) == 0
    # heads that fill the SMs many times over need no partial sums
    assert W(64, 64, 64, 1, 1500, 64, 1) == 0 or W(64, 64, 64, 1, 1500, 64, 1) < 1 << 20
    assert W(256, 64, 64, 300, 500, 64, 1) == 0
    assert W(1, 1, 1, 1, 100, 64, 1) == 0 and W(1, 1, 1, 1, 100000, 64, 1) > 0
    # the partial sums of the tensor cores are bounded by the grid, not by the problem
    assert W(1, 8, 8, 8192, 16384, 64, 1) <= 148 * 2 * 128 * 65 * 4 + 65536
    assert V(1, 8, 8, 8192, 16384, 64, 1) >= 2 * 8 * 8192 * 4


def test_binding_refuses_before_the_library():
    import torch

    kbuild.build()
    K = E
    x = torch.zeros(1, 2, 3, 16)
    with pytest.raises(K.KataError, match="must be a CUDA tensor"):
        K.kata_cross_forward(x, x, x)
    with pytest.raises(K.KataError, match="must be a CUDA tensor"):
        K.kata_qk_norm_rotate(x)
