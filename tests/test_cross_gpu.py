"""kata_cross_forward and kata_cross_backward against the 64-bit forms (tests/layer_oracle.py)."""
from __future__ import annotations

import pytest

from tests import layer_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import kernelized_linear_attention_fwd_b200 as K  # noqa: E402
from kernelized_linear_attention_fwd_b200.csrc import build as kbuild  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    K.load_library()
    yield
    assert K.kata_get_device_status() == 0


def make(B, H, Hk, Tq, Tk, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, device="cuda", generator=g)

    def unit(x):
        return x / (x * x).mean(-1, keepdim=True).sqrt()

    dt = DT[dtype]
    return (unit(r(B, H, Tq, d)).to(dt), unit(r(B, Hk, Tk, d)).to(dt), r(B, Hk, Tk, d).to(dt),
            r(B, H, Tq, d).to(dt))


def lens(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


def forward(q, k, v, n):
    y = torch.full(q.shape, float("nan"), device="cuda")
    den = torch.full(q.shape[:3], float("nan"), device="cuda")
    out = K.kata_cross_forward(q, k, v, key_lengths=n, y_out=y, den_out=den)
    return out, y, den


def check(q, k, v, g, n=None, backward=True):
    out, y, den = forward(q, k, v, n)
    ry, rl = O.cross(q, k, v, n)
    bo, by = O.cross_bounds(q, k, v, q.dtype, n)
    assert O.worst(out, ry, bo) <= 1
    assert O.worst(y, ry, by) <= 1
    e = O.HALF[q.dtype] if q.dtype == torch.bfloat16 else 0.0
    assert float(((den.double() - rl).abs() / (rl + 1e-30)).max()) <= 1.1 * e + 1e-3 * O.HALF[torch.bfloat16] * 16
    if not backward:
        return
    got = K.kata_cross_backward(g, q, k, v, y, den, key_lengths=n)
    ref = O.cross_grad(g, q, k, v, n)
    bounds = O.cross_bounds(q, k, v, q.dtype, n, dout=g)
    for name, a, r, b in zip(("dq", "dk", "dv"), got, ref, bounds):
        w = O.worst(a, r, b)
        assert w <= 1, f"{name}: {w:.2f} of its bound"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("Tq,Tk", [(1, 1), (1, 300), (63, 65), (129, 64), (200, 333)])
def test_head_sizes_and_lengths(dtype, d, Tq, Tk):
    check(*make(2, 2, 2, Tq, Tk, d, dtype, seed=d + Tq))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk", [(255, 127), (256, 128), (257, 129), (1, 2049), (385, 513), (700, 900)])
def test_around_the_tiles(dtype, Tq, Tk):
    check(*make(1, 2, 1, Tq, Tk, 64, dtype, seed=Tq))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padded_batch_with_empty_and_single_key_rows(dtype):
    for Tk in (70, 128, 300):
        q, k, v, g = make(6, 4, 2, 45, Tk, 64, dtype, seed=Tk)
        n = lens(Tk, 0, 1, 64, Tk - 1, 17)
        check(q, k, v, g, n)
        out, y, den = forward(q, k, v, n)
        dq, dk, dv = K.kata_cross_backward(g, q, k, v, y, den, key_lengths=n)
        assert float(out[1].abs().max()) == 0 and float(dq[1].abs().max()) == 0
        assert float(dk[1].abs().max()) == 0 and float(dv[1].abs().max()) == 0
        for b in range(6):
            assert not dk[b, :, int(n[b]):].any() and not dv[b, :, int(n[b]):].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_visible_key(dtype):
    # y = v and the gradients of q and k vanish (the weights cancel)
    q, k, v, g = make(2, 2, 2, 33, 200, 64, dtype, seed=3)
    n = lens(1, 1)
    out, y, den = forward(q, k, v, n)
    assert O.worst(y, v[:, :, :1].double().expand(-1, -1, 33, -1), 4 * O.U * v[:, :, :1].double().abs() + 1e-30) <= 1
    dq, dk, _ = K.kata_cross_backward(g, q, k, v, y, den, key_lengths=n)
    s = (q.double() * k[:, :, :1].double()).sum(-1, keepdim=True)
    P = (g.double().abs() * v[:, :, :1].double().abs()).sum(-1, keepdim=True)
    # c = 2 (p - D) / s with p - D below 80 U P, s itself off by up to e in 1 / l
    c = 1.1 * 2 * 80 * O.U * P / s.abs()
    assert float((dq.double().abs() / (c * k[:, :, :1].double().abs() + 1e-30)).max()) <= 1
    assert float((dk[:, :, 0].double().abs() / ((c * q.double().abs()).sum(2) + 1e-30)).max()) <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), "lowest"])
def test_what_masked_keys_hold_does_not_matter(dtype, bad):
    for n in (lens(77, 0, 130), lens(128, 1, 64)):
        q, k, v, g = make(3, 4, 2, 50, 300, 64, dtype, seed=8)
        value = torch.finfo(q.dtype).min if bad == "lowest" else bad
        out, y, den = forward(q, k, v, n)
        ref = (out, y, den) + K.kata_cross_backward(g, q, k, v, y, den, key_lengths=n)
        k2, v2 = k.clone(), v.clone()
        for b in range(3):
            k2[b, :, int(n[b]):] = value
            v2[b, :, int(n[b]):] = value
        out, y, den = forward(q, k2, v2, n)
        got = (out, y, den) + K.kata_cross_backward(g, q, k2, v2, y, den, key_lengths=n)
        for a, b in zip(ref, got):
            assert torch.equal(a, b)


def test_lengths_outside_the_range_are_clamped():
    q, k, v, g = make(3, 2, 2, 20, 100, 32, "bf16", seed=4)
    a = forward(q, k, v, lens(-5, 1000, 100))
    b = forward(q, k, v, lens(0, 100, 100))
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_orthogonal_queries_have_no_weight(dtype):
    q, k, v, g = make(1, 1, 1, 40, 90, 64, dtype, seed=5)
    q[..., 32:] = 0
    k[..., :32] = 0
    out, y, den = forward(q, k, v, None)
    grads = K.kata_cross_backward(g, q, k, v, y, den)
    for t in (out, y, den) + grads:
        assert not t.any()


@pytest.mark.parametrize("H,Hk", [(1, 1), (8, 1), (12, 3), (16, 16)])
def test_shared_key_heads(H, Hk):
    for dtype in ("bf16", "f32"):
        check(*make(2, H, Hk, 70, 150, 32, dtype, seed=H))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,Tk", [(1, 8, 2, 20000), (2, 2, 2, 4097), (1, 1, 1, 66000)])
def test_single_token_against_a_long_memory(dtype, B, H, Hk, Tk):
    # the keys are split over the SMs and joined
    q, k, v, g = make(B, H, Hk, 1, Tk, 64, dtype, seed=Tk)
    code = 1 if dtype == "bf16" else 0
    assert K.kata_cross_forward_workspace_bytes(B, H, Hk, 1, Tk, 64, code) > 0
    check(q, k, v, g)
    check(q, k, v, g, torch.randint(1, Tk, (B,), device="cuda").int())


@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("H,Hk,Tq,Tk", [(5, 1, 1, 3000), (8, 1, 1, 1), (16, 2, 1, 20000), (16, 1, 1, 127), (6, 3, 4, 129),
                                        (2, 2, 13, 16), (3, 3, 16, 700), (17, 1, 1, 900), (2, 2, 32, 5000)])
def test_steps_of_several_rows(H, Hk, Tq, Tk, d):
    # up to 32 rows a key head in bf16: errors are the outputs' rounding
    q, k, v, g = make(3, H, Hk, Tq, Tk, d, "bf16", seed=Tk + d)
    for n in (None, lens(Tk, 0, (Tk + 1) // 2)):
        kk, vv = k.clone(), v.clone()
        if n is not None:
            for b in range(3):
                kk[b, :, int(n[b]):], vv[b, :, int(n[b]):] = float("nan"), float("inf")
        out, y, den = forward(q, kk, vv, n)
        ref, l = O.cross(q, k, v, n)
        bo, by = O.cross_bounds(q, k, v, q.dtype, n, split=True)
        assert O.worst(out, ref, bo) <= 1 and O.worst(y, ref, by) <= 1
        # without the exports the same kernel
        assert torch.equal(out, K.kata_cross_forward(q, kk, vv, key_lengths=n))
    check(q, k, v, g, lens(Tk, 0, (Tk + 1) // 2))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_queries_on_few_keys(dtype):
    # the queries are split over the SMs for dk and dv
    q, k, v, g = make(1, 4, 1, 3000, 40, 64, dtype, seed=6)
    assert K.kata_cross_backward_workspace_bytes(1, 4, 1, 3000, 40, 64, 1 if dtype == "bf16" else 0) > 0
    check(q, k, v, g)


def test_many_items_of_one_and_two_tiles():
    # several items per SM: single tiles alternate between the two halves
    check(*make(40, 8, 8, 100, 200, 32, "bf16", seed=7))
    q, k, v, g = make(64, 6, 6, 140, 140, 16, "bf16", seed=9)
    check(q, k, v, g, torch.randint(0, 141, (64,), device="cuda").int())


@pytest.mark.parametrize("scale", [2.0 ** -12, 2.0 ** 12])
def test_scales_of_queries_and_keys_cancel(scale):
    for dtype in ("bf16", "f32"):
        q, k, v, g = make(1, 2, 2, 65, 130, 64, dtype, seed=12)
        a = K.kata_cross_forward(q, k, v)
        b = K.kata_cross_forward(q * scale, k * scale, v)
        assert torch.equal(a, b)  # powers of two: the same bits


def test_gradient_against_differences():
    q, k, v, g = make(2, 4, 2, 5, 9, 16, "f32", seed=13)
    n = lens(9, 4)
    _, y, den = forward(q, k, v, n)
    grads = K.kata_cross_backward(g, q, k, v, y, den, key_lengths=n)
    bounds = O.cross_bounds(q, k, v, torch.float32, n, dout=g)
    h = 1e-6
    for seed in range(4):
        gg = torch.Generator(device="cuda").manual_seed(seed)
        dirs = [torch.randn(t.shape, device="cuda", generator=gg).double() for t in (q, k, v)]

        def f(sign):
            t = [x.double() + sign * h * e for x, e in zip((q, k, v), dirs)]
            return float((O.cross(*t, n)[0] * g.double()).sum())

        num = (f(1) - f(-1)) / (2 * h)
        ana = sum(float((a.double() * e).sum()) for a, e in zip(grads, dirs))
        tol = sum(float((b * e.abs()).sum()) for b, e in zip(bounds, dirs))
        scale = sum(float((a.double() * e).abs().sum()) for a, e in zip(grads, dirs))
        assert abs(num - ana) <= tol + 1e-7 * scale


@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("H,Hk,Tq,Tk", [(2, 2, 300, 1), (2, 1, 1, 2), (4, 2, 16, 5), (3, 3, 700, 9), (8, 8, 130, 32),
                                        (2, 2, 32, 1000), (4, 1, 8, 300), (1, 1, 1, 4097), (6, 3, 5, 130)])
def test_few_terms_keep_their_precision(H, Hk, Tq, Tk, d):
    # the operands go back as two bf16 numbers: only the outputs' rounding is left
    q, k, v, g = make(2, H, Hk, Tq, Tk, d, "bf16", Tq + Tk)
    n = lens(Tk, max(1, Tk // 2))
    y, den = forward(q, k, v, n)[1:]
    got = K.kata_cross_backward(g, q, k, v, y, den, key_lengths=n)
    for a, r, b in zip(got, O.cross_grad(g, q, k, v, n), O.cross_bounds(q, k, v, q.dtype, n, dout=g, split=True)):
        assert O.worst(a, r, b) <= 1


def test_few_terms_with_masked_keys_of_any_content():
    q, k, v, g = make(3, 4, 2, 70, 29, 64, "bf16", 5)
    n = lens(17, 0, 1)
    for b, x in enumerate((17, 0, 1)):
        k[b, :, x:], v[b, :, x:] = float("nan"), float("-inf")
    out, y, den = forward(q, k, v, n)
    got = K.kata_cross_backward(g, q, k, v, y, den, key_lengths=n)
    kk, vv = k.clone(), v.clone()
    for b, x in enumerate((17, 0, 1)):
        kk[b, :, x:], vv[b, :, x:] = 0, 0
    assert not out[1].any() and not got[0][1].any()
    for a, r, b in zip(got, O.cross_grad(g, q, kk, vv, n), O.cross_bounds(q, kk, vv, q.dtype, n, dout=g, split=True)):
        assert O.worst(a, r, b) <= 1


@pytest.mark.parametrize("Tq,Tk", [(257, 700), (40, 4000), (1000, 33)])
def test_query_gradient_of_the_smallest_heads_keeps_its_precision(Tq, Tk):
    q, k, v, g = make(2, 4, 2, Tq, Tk, 16, "bf16", Tq)
    n = lens(Tk, Tk // 3)
    y, den = forward(q, k, v, n)[1:]
    dq = K.kata_cross_backward(g, q, k, v, y, den, key_lengths=n)[0]
    bound = O.cross_bounds(q, k, v, q.dtype, n, dout=g, split=True)[0]
    assert O.worst(dq, O.cross_grad(g, q, k, v, n)[0], bound) <= 1


def test_outputs_are_convex_combinations():
    q, k, v, _ = make(1, 2, 2, 100, 400, 64, "bf16", seed=14)
    _, y, _ = forward(q, k, v, None)
    lo, hi = v.float().amin(2, keepdim=True), v.float().amax(2, keepdim=True)
    assert bool((y >= lo - 1e-5).all()) and bool((y <= hi + 1e-5).all())


def test_same_bits_on_a_second_call():
    q, k, v, g = make(1, 4, 1, 1000, 3000, 64, "bf16", seed=15)
    a, b = forward(q, k, v, None), forward(q, k, v, None)
    ga = K.kata_cross_backward(g, q, k, v, a[1], a[2])
    gb = K.kata_cross_backward(g, q, k, v, b[1], b[2])
    for x, y in zip(a + ga, b + gb):
        assert torch.equal(x, y)
