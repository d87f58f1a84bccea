"""fp32 cross attention keeps fp32 accuracy: the root mean square of each output's error.

The elementwise bounds of tests/layer_oracle.py hold for the worst signs and are some
hundred times what comes out; a kernel that kept 16 bits of its operands instead of 24
would pass many of them.  The limit here, LIMIT = 8 U (U = 2^-24) of the output's root mean
square, for inputs of random signs: a product of the kernels is off by at most 2 U of its
result's root mean square (few additions at the result's own size: a head's 64 coordinates
in 4, a block's 64 columns in 4, up to 64 blocks, whose partial sums grow with the
root of their number: U sqrt(64 / 6) = 3.3 U at worst, 2 U at half of that).  The weights, squares of a product, are then
off by 4 U, what they weigh by another 2 to 3, a quotient by 1; roundings add as squares,
so below 6 U for y and l.  c = 2 s (p - D) / l: s and p 2 U each, D 3, 1 / l 4: below 6 U, with
the gradients' own sums below 7 U.  Operands of two bf16 parts lose 2^-17 of an operand at most,
2^-17 / sqrt(3) = 4.4e-6 root mean square of the last digit's range, 9 times the limit
before anything adds up (the first test takes them through the 64-bit form).
"""
from __future__ import annotations

import pytest

from tests import layer_oracle as O

torch = pytest.importorskip("torch")

LIMIT = 8 * O.U
NAMES = ("out", "y", "den", "dq", "dk", "dv")


def make(B, H, Hk, Tq, Tk, d, seed, device):
    g = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g)

    def unit(x):
        return x / (x * x).mean(-1, keepdim=True).sqrt()

    t = unit(r(B, H, Tq, d)), unit(r(B, Hk, Tk, d)), r(B, Hk, Tk, d), r(B, H, Tq, d)
    return [x.to(device) for x in t]


def rms(got, want):
    want = want.double()
    return float((got.double() - want).pow(2).mean().sqrt() / want.pow(2).mean().sqrt())


def cut(x, parts):
    """x as the sum of its first bf16 parts."""
    total = torch.zeros_like(x)
    for _ in range(parts):
        total = total + (x - total).bfloat16().to(x.dtype)
    return total


@pytest.mark.parametrize("shape", [(1, 2, 2, 100, 200, 64), (2, 2, 1, 40, 300, 16)])
def test_the_limit_tells_two_parts_from_three(shape):
    q, k, v, g = (x.double() for x in make(*shape, 1, "cpu"))
    q, k, v, g = (x.float().double() for x in (q, k, v, g))
    exact = O.cross(q, k, v) + O.cross_grad(g, q, k, v)
    # every product with operands of two parts, or the value products and gradient sums alone
    cq, ck, cv, cg = (cut(x, 2) for x in (q, k, v, g))
    for got in (O.cross(cq, ck, cv) + O.cross_grad(cg, cq, ck, cv),
                (O.cross(q, k, cv)[0], O.cross(cq, k, v)[1], O.cross_grad(g, q, ck, v)[0],
                 O.cross_grad(g, cq, k, v)[1], O.cross_grad(cg, q, k, v)[2])):
        for name, a, b in zip(("y", "den", "dq", "dk", "dv"), got, exact):
            assert rms(a, b) > 2 * LIMIT, name
    kept = [cut(x, 3) for x in (q, k, v, g)]
    for a, b in zip(O.cross(*kept[:3]) + O.cross_grad(kept[3], *kept[:3]), exact):
        assert rms(a, b) < 0.1 * LIMIT


# whole tiles and ragged ones, shared key heads, pieces of the keys or of the queries joined,
# steps of 1, 2 and 4 rows on the CUDA cores and of 5 to 32 by products
SHAPES = [(2, 2, 2, 129, 200, 16), (2, 2, 2, 200, 333, 32), (1, 4, 2, 301, 517, 64), (1, 8, 8, 700, 900, 64),
          (1, 1, 1, 64, 4000, 64), (1, 2, 1, 2500, 70, 64), (64, 8, 8, 100, 130, 32), (3, 2, 2, 1, 2049, 64),
          (2, 4, 2, 1, 3000, 32), (2, 4, 1, 1, 700, 64), (2, 8, 1, 1, 900, 16), (1, 2, 2, 17, 3000, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("padded", [False, True])
def test_root_mean_square_errors(shape, padded):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import kernelized_linear_attention_fwd_b200 as K

    B, H, Hk, Tq, Tk, d = shape
    q, k, v, g = make(*shape, Tq + Tk, "cuda")
    n = None
    if padded:
        n = torch.tensor([Tk - b * Tk // (2 * B) - 1 for b in range(B)], dtype=torch.int32, device="cuda")
    y, den = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:3], device="cuda")
    out = K.kata_cross_forward(q, k, v, key_lengths=n, y_out=y, den_out=den)
    got = (out, y, den) + K.kata_cross_backward(g, q, k, v, y, den, key_lengths=n)
    ry, rl = O.cross(q, k, v, n)
    for name, a, b in zip(NAMES, got, (ry, ry, rl) + O.cross_grad(g, q, k, v, n)):
        assert rms(a, b) <= LIMIT, (name, rms(a, b) / O.U)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
def test_denominators_within_the_rounding_of_their_sum(shape):
    # l = sum s^2: a product off by a A (A = sum |q_i k_i|, a of cross_bounds) enters as 2 |s| a A,
    # and the sum of positive terms rounds by a of itself
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import kernelized_linear_attention_fwd_b200 as K

    B, H, Hk, Tq, Tk, d = shape
    q, k, v, _ = make(*shape, 3 + Tk, "cuda")
    den = torch.empty(q.shape[:3], device="cuda")
    K.kata_cross_forward(q, k, v, den_out=den)
    qq, kk = q.double().reshape(B, Hk, -1, d), k.double().transpose(-1, -2)
    s, A = qq @ kk, qq.abs() @ kk.abs()
    a = O.U * (64 + 8 + max(Tk, qq.shape[2]) / 64)
    bound = 1.1 * a * (2 * (s.abs() * A).sum(-1) + (s * s).sum(-1))
    assert float(((den.double() - (s * s).sum(-1).reshape(den.shape)).abs() / bound.reshape(den.shape)).max()) <= 1
