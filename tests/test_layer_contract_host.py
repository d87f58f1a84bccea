"""Host-side promises of the head norm's and cross attention's entry points (no GPU).  As
in tests/test_layer_abi_host.py every call passes fake addresses and is refused; what an
accepted call is refused for, last of all, is its missing workspace (WS)."""
import glob
import itertools
import os
import random
import re

import pytest

from kernelized_linear_attention_fwd_b200.csrc import build as kbuild
from tests.test_layer_abi_host import INV, UNS, WS, at, lib, norm, norm_bwd  # noqa: F401  (lib: a fixture)


# ------------------------------------------------------- dq and dk in one buffer

def grads(lib, n, dq, dk, gap, H=(1, 1), d=16):
    """The status of a gradient whose dq and dk have these strides, dk `gap` elements
    behind dq (bf16), with no workspace: WS once the layout is taken."""
    B, T = n
    return norm_bwd(lib, B=B, T=T, Hq=H[0], Hk=H[1], d=d, n=0, inv=0, pos=0, qs=(0, 0, 0), ks=(0, 0, 0), dqs=dq,
                    dks=dk, dk=at(8, 2 * gap), ws=0)


def rows_meet(n, dq, dk, gap, H, d):
    """Whether any element belongs to two rows, by listing the rows' first elements."""
    starts = [b * s[0] + t * s[1] + h * s[2] + o
              for s, heads, o in ((dq, H[0], 0), (dk, H[1], gap))
              for b, t, h in itertools.product(range(n[0]), range(n[1]), range(heads))]
    starts.sort()
    return any(y - x < d for x, y in zip(starts, starts[1:]))


def test_overlapping_gradients_are_refused(lib):
    # dk lies one token behind dq: dq of (1, 0) and dk of (0, 1) are the same row
    assert grads(lib, (2, 2), (192, 128, 64), (192, 128, 64), 64, d=64) == INV
    # dk's second sequence inside dq's third
    assert grads(lib, (3, 1), (32, 16, 16), (32, 16, 16), 64) == INV


@pytest.mark.parametrize("B", [1, 3])
@pytest.mark.parametrize("H", [(4, 2), (1, 4), (4, 1), (1, 1)])
def test_slices_of_one_buffer_are_taken_in_every_order(lib, B, H):
    T, d, n = 5, 16, H[0] + H[1] + 2
    token = (T * n * d, n * d, d)          # [B, T, H, d]
    head = (n * T * d, d, T * d)           # [B, H, T, d]
    first = (n * d, B * n * d, d)          # [T, B, H, d]
    for s, step in ((token, d), (head, T * d), (first, d)):
        assert grads(lib, (B, T), s, s, H[0] * step, H, d) == WS
        assert grads(lib, (B, T), s, s, (H[0] + 2) * step, H, d) == WS
        if H[0] > 1 or T > 1:
            assert grads(lib, (B, T), s, s, (H[0] - 1) * step, H, d) == INV
    # heads of queries, keys and values in turn: [B, T, H, 3, d]
    s = (T * 12 * d, 12 * d, 3 * d)
    assert grads(lib, (B, T), s, s, d, H, d) == WS
    # dk token by token where dq leaves room, dq and dk of other steps
    assert grads(lib, (B, T), (T * 32 * d, 32 * d, d), (T * 32 * d, 32 * d, 2 * d), 8 * d, H, d) == WS
    # apart
    assert grads(lib, (B, T), token, head, B * T * n * d, H, d) == WS


def test_a_layout_is_taken_only_without_a_shared_element(lib):
    rng = random.Random(5)
    taken = 0
    for _ in range(20000):
        n = rng.choice([1, 2, 3]), rng.choice([1, 2, 3])
        H = rng.choice([1, 2, 3]), rng.choice([1, 2, 3])
        dq = [8 * rng.randrange(0, 25) for _ in range(3)]
        dk = list(dq) if rng.random() < 0.7 else [8 * rng.randrange(0, 25) for _ in range(3)]
        gap = 8 * rng.randrange(0, 40)
        if grads(lib, n, dq, dk, gap, H) == WS:
            taken += 1
            assert not rows_meet(n, dq, dk, gap, H, 16), (n, H, dq, dk, gap)
    assert taken > 500


# ------------------------------------------------------------------ head counts

def test_head_counts_near_2_to_31_are_refused(lib):
    # the set counts of a block row would pass 2^31
    W = lib.kata_qk_norm_rotate_backward_workspace_bytes
    top = 2 ** 31 - 2 ** 17
    for d in (16, 32, 64):
        assert W(1, 1, top - 1, 1, d) > 0 and W(1, 1, 1, top - 1, d) > 0
        for n in (top, 2 ** 31 - 64, 2 ** 31 - 1):
            assert W(1, 1, n, 1, d) == 0 and W(1, 1, 1, n, d) == 0
    far = dict(B=1, T=1, qs=(0, 0, 64), ks=(0, 0, 64), dqs=(0, 0, 64), dks=(0, 0, 64))
    for bad in (dict(Hq=top), dict(Hk=top), dict(Hq=2 ** 31 - 1), dict(Hk=2 ** 31 - 1)):
        assert norm(lib, **{k: x for k, x in far.items() if k[0] != "d"}, **bad) == UNS
        assert norm_bwd(lib, **far, **bad) == UNS


# ---------------------------------------------------------- alignment of arrays

SIZES = {"float": 4, "int": 4, "uint32_t": 4, "uint16_t": 2, "uint8_t": 1, "float2": 8, "uint2": 8, "uint64_t": 8,
         "float4": 16, "uint4": 16}
ARRAY = re.compile(r"(__shared__\s+)?(?:alignas|__align__)?(\(\d+\))?\s*\b(%s)\s+([^;=()]*\[[^;=()]*)[;=]" % "|".join(SIZES))
CAST = re.compile(r"reinterpret_cast<(?:const )?(float2|uint2|uint64_t|float4|uint4) \*>\(&?(\w+)\b")


def under_aligned(source):
    """Names of arrays that are read or written as vectors wider than they are aligned, function by
    function (a function opens at a line that starts with a brace's head and ends at `}` in column 0)."""
    found = []
    for body in re.split(r"(?m)^\}", source):
        align = {}
        for m in ARRAY.finditer(body):
            a = int(m.group(2)[1:-1]) if m.group(2) else SIZES[m.group(3)]
            for name in re.findall(r"(\w+)(?:\[[^\]]*\])+", m.group(4)):
                align[name] = a
        found += [m.group(2) for m in CAST.finditer(body) if align.get(m.group(2), 16) < SIZES[m.group(1)]]
    return found


def test_arrays_read_as_vectors_are_aligned_for_it():
    bad = "__global__ void f() {\n    __shared__ float a[4][8], b[2];\n    *reinterpret_cast<float4 *>(&a[i][4]) = x;\n}\n"
    assert under_aligned(bad) == ["a"]
    assert under_aligned(bad.replace("float a[", "__align__(16) float a[")) == []
    for path in sorted(glob.glob(os.path.join(kbuild.HERE, "*.cu*"))):
        with open(path) as f:
            assert under_aligned(f.read()) == [], os.path.basename(path)
