"""kata_qk_norm_rotate and its gradient against the 64-bit forms (tests/layer_oracle.py)."""
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make(B, T, H, Hk, d, dtype, seed, fused=True):
    g = gen(seed)
    n = H + 2 * Hk + 1 if fused else H + Hk
    proj = torch.randn(B, T, n, d, device="cuda", generator=g)
    proj = (proj * torch.exp(torch.randn(B, T, n, 1, device="cuda", generator=g))).to(DT[dtype])
    return proj, proj[:, :, :H], proj[:, :, H:H + Hk] if Hk else None


def freq(n):
    return (10000.0 ** (-torch.arange(n, device="cuda").double() / max(1, n))).float()


def check(B, T, H, Hk, d, dtype, n, inter, seed, pos="far", weights=True):
    g = gen(seed + 1)
    _, q, k = make(B, T, H, Hk, d, dtype, seed)
    wq = 1 + 0.3 * torch.randn(d, device="cuda", generator=g) if weights else None
    wk = 1 + 0.3 * torch.randn(d, device="cuda", generator=g) if weights and Hk else None
    inv = freq(n) if n else None
    if pos == "far":
        p = torch.randint(0, 2 ** 24, (B, T), device="cuda", generator=g)
    elif pos == "shared":
        p = torch.randint(0, 2 ** 17, (T,), device="cuda", generator=g)
    else:
        p = None
    kw = dict(q_weight=wq, k_weight=wk, inv_freq=inv, positions=p, eps=1e-5, interleaved=inter)
    yq, yk = K.kata_qk_norm_rotate(q, k, **kw)
    ang = O.angles(p, inv, B, T, "cuda")
    gq = torch.randn(yq.shape, device="cuda", generator=g).to(q.dtype)
    gk = torch.randn(yk.shape, device="cuda", generator=g).to(q.dtype) if Hk else None
    dq, dk, dwq, dwk = K.kata_qk_norm_rotate_backward(gq, gk, q, k, **kw)
    for y, x, w, gy, dx, dw in ((yq, q, wq, gq, dq, dwq), (yk, k, wk, gk, dk, dwk)):
        if x is None:
            assert y is None and dx is None and dw is None
            continue
        ref = O.norm_rotate(x, w, ang, 1e-5, inter)
        assert O.worst(y, ref, O.norm_rotate_bounds(ref, x, w, x.dtype, 1e-5, inter, n)) <= 1
        rdx, rdw = O.norm_rotate_grad(gy, x, w, ang, 1e-5, inter)
        bdx, bdw = O.norm_grad_bounds(rdx, gy, x, w, x.dtype, 1e-5, inter, n)
        assert O.worst(dx, rdx, bdx) <= 1
        assert O.worst(dw, rdw, bdw) <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,n", [(16, 8), (16, 4), (32, 16), (32, 12), (64, 32), (64, 4), (64, 0)])
def test_head_sizes_and_partial_rotation(dtype, inter, d, n):
    check(2, 37, 5, 3, d, dtype, n, inter, seed=d + n)


@pytest.mark.parametrize("n", [1, 3, 5, 31])
def test_odd_numbers_of_interleaved_pairs(n):
    check(1, 9, 2, 2, 64, "f32", n, True, seed=n)


@pytest.mark.parametrize("B,T,H,Hk", [(1, 1, 1, 1), (64, 1, 16, 16), (3, 1, 16, 1), (1, 2, 33, 1), (1, 4099, 2, 1),
                                      (5, 7, 1, 0), (2, 130, 64, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shapes(B, T, H, Hk, dtype):
    check(B, T, H, Hk, 64, dtype, 32, False, seed=B + T)


@pytest.mark.parametrize("d,H,Hk", [(64, 2, 1), (64, 3, 2), (64, 4, 0), (64, 4, 8), (64, 9, 2), (64, 15, 15), (64, 5, 16),
                                    (32, 1, 2), (32, 7, 3), (32, 16, 9), (32, 31, 4), (16, 1, 1), (16, 9, 2), (16, 17, 3),
                                    (16, 63, 1)])
@pytest.mark.parametrize("dtype,inter", [("bf16", True), ("f32", False)])
def test_head_counts_about_a_warps_rows(d, H, Hk, dtype, inter):
    # tokens that end inside a warp's, batches that end inside them, several turns of a warp
    check(3, 67, H, Hk, d, dtype, d // 2, inter, seed=H + Hk)
    check(1, 2371 * 64 // d + 1, H, Hk, d, dtype, d // 4, inter, seed=H + Hk + 1)


def test_no_gain_and_default_positions():
    check(2, 70, 3, 2, 32, "f32", 16, False, seed=5, pos=None, weights=False)


def test_positions_shared_by_the_batch():
    check(3, 70, 3, 2, 32, "bf16", 16, True, seed=6, pos="shared")


def test_far_positions():
    # 2^31 + small: the fraction of a turn keeps 2^-22 of a turn, 1.5e-6 rad
    q = make(1, 4, 2, 0, 64, "f32", 9)[1]
    p = torch.tensor([[2 ** 31, 2 ** 31 + 1, 2 ** 31 + 77, 5]], device="cuda")
    y, _ = K.kata_qk_norm_rotate(q, inv_freq=freq(32), positions=p)
    ref = O.norm_rotate(q, None, O.angles(p, freq(32), 1, 4, "cuda"), 1e-6, False)
    assert float((y.double() - ref).abs().max()) <= 4e-6 * float(ref.abs().max())


def test_rows_of_zeros_give_zeros():
    q = torch.zeros(1, 3, 2, 32, device="cuda")
    y, _ = K.kata_qk_norm_rotate(q, inv_freq=freq(16))
    assert float(y.abs().max()) == 0
    g = torch.ones(1, 2, 3, 32, device="cuda")
    dq, _, dw, _ = K.kata_qk_norm_rotate_backward(g, None, q, inv_freq=freq(16))
    assert torch.isfinite(dq).all() and float(dw.abs().max()) == 0


def test_a_bad_row_stays_in_its_row():
    q = make(1, 40, 4, 0, 64, "f32", 11)[1].clone()
    y0, _ = K.kata_qk_norm_rotate(q, inv_freq=freq(32))
    q[0, 7, 2, 5] = float("nan")
    q[0, 8, 1, 5] = float("inf")
    y1, _ = K.kata_qk_norm_rotate(q, inv_freq=freq(32))
    keep = torch.ones(1, 4, 40, dtype=torch.bool, device="cuda")
    keep[0, 2, 7] = keep[0, 1, 8] = False
    assert torch.equal(y0[keep], y1[keep]) and torch.isnan(y1[0, 2, 7]).all()


def test_strided_inputs_and_fused_gradient():
    B, T, H, Hk, d = 2, 33, 4, 2, 32
    proj, q, k = make(B, T, H, Hk, d, "bf16", 21)
    kw = dict(inv_freq=freq(16))
    a = K.kata_qk_norm_rotate(q, k, **kw)
    b = K.kata_qk_norm_rotate(q.contiguous(), k.contiguous(), **kw)
    # head-major storage seen as token-major: other strides, same values
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    c = K.kata_qk_norm_rotate(qt, k, **kw)
    for x in (b, c):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])
    gq, gk = torch.randn_like(a[0]), torch.randn_like(a[1])
    fused = torch.full_like(proj, 7.0)
    K.kata_qk_norm_rotate_backward(gq, gk, q, k, dq=fused[:, :, :H], dk=fused[:, :, H:H + Hk], **kw)
    dq, dk, _, _ = K.kata_qk_norm_rotate_backward(gq, gk, q, k, **kw)
    assert torch.equal(fused[:, :, :H], dq) and torch.equal(fused[:, :, H:H + Hk], dk)
    assert bool((fused[:, :, H + Hk:] == 7.0).all())  # the values' part as it was
    # one sequence broadcast over the batch (stride 0) as input
    e = q[:1].expand(3, -1, -1, -1)
    assert torch.equal(K.kata_qk_norm_rotate(e, **kw)[0][2], a[0][0])


def test_gradient_against_differences():
    B, T, H, d = 1, 6, 2, 16
    _, q, _ = make(B, T, H, 0, d, "f32", 31)
    g = gen(32)
    w = 1 + 0.3 * torch.randn(d, device="cuda", generator=g)
    p = torch.randint(0, 1000, (B, T), device="cuda", generator=g)
    gy = torch.randn(B, H, T, d, device="cuda", generator=g)
    dq, _, dw, _ = K.kata_qk_norm_rotate_backward(gy, None, q, q_weight=w, inv_freq=freq(8), positions=p)
    ang = O.angles(p, freq(8), B, T, "cuda")

    def f(x, ww):
        return float((O.norm_rotate(x, ww, ang, 1e-6, False) * gy.double()).sum())

    h = 1e-5
    for seed in range(3):
        dx = torch.randn(q.shape, device="cuda", generator=gen(seed)).double()
        dd = torch.randn(d, device="cuda", generator=gen(seed + 9)).double()
        num = (f(q.double() + h * dx, w.double() + h * dd) - f(q.double() - h * dx, w.double() - h * dd)) / (2 * h)
        ana = float((dq.double() * dx).sum() + (dw.double() * dd).sum())
        scale = float((dq.double() * dx).abs().sum() + (dw.double() * dd).abs().sum())
        # fp32 gradients: 100 U of the magnitudes; differences: h^2 of third derivatives
        assert abs(num - ana) <= 100 * O.U * scale + 1e-6 * scale


def test_same_bits_on_a_second_call_and_given_buffers():
    _, q, k = make(2, 300, 4, 4, 64, "bf16", 41)
    kw = dict(inv_freq=freq(32))
    yq, yk = K.kata_qk_norm_rotate(q, k, **kw)
    gq, gk = torch.randn_like(yq), torch.randn_like(yk)
    a = K.kata_qk_norm_rotate_backward(gq, gk, q, k, **kw)
    ws = torch.full((K.kata_qk_norm_rotate_backward_workspace_bytes(2, 300, 4, 4, 64) + 256,), 255,
                    dtype=torch.uint8, device="cuda")[:-256]
    dw = torch.full((64,), float("nan"), device="cuda")
    b = K.kata_qk_norm_rotate_backward(gq, gk, q, k, workspace=ws, dq_weight=dw, **kw)
    assert b[2] is dw
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_offsets_past_32_bits():
    # a token stride that puts the last rows past 2^32 bytes and 2^31 elements
    T, st = 5, 2 ** 29 + 64
    buf = torch.zeros((T - 1) * st + 64, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(1, T, 1, 64, device="cuda").to(torch.bfloat16)
    q = buf.as_strided((1, T, 1, 64), (0, st, 64, 1))
    q.copy_(x)
    y, _ = K.kata_qk_norm_rotate(q, inv_freq=freq(32))
    assert torch.equal(y, K.kata_qk_norm_rotate(x, inv_freq=freq(32))[0])
    dq = torch.zeros_like(buf).as_strided(q.shape, q.stride())
    a = K.kata_qk_norm_rotate_backward(y, None, q, inv_freq=freq(32), dq=dq)[0]
    assert torch.equal(a, K.kata_qk_norm_rotate_backward(y, None, x, inv_freq=freq(32))[0])
