"""What include/kata.h promises of the head norm and of cross attention beyond their
values on ordinary inputs: layouts of the gradients, zeros behind the last key whatever
the queries hold."""
from __future__ import annotations

import pytest

from tests import layer_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import kernelized_linear_attention_fwd_b200 as K  # noqa: E402
from kernelized_linear_attention_fwd_b200.csrc import build as kbuild  # noqa: E402
from tests.test_cross_gpu import forward, lens, make  # noqa: E402
from tests.test_norm_rotate_gpu import freq  # noqa: E402
from tests.test_norm_rotate_gpu import make as norm_make  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    K.load_library()
    yield
    assert K.kata_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk", [(4, 2), (1, 1), (16, 4)])
def test_gradients_as_slices_of_one_buffer_in_any_order(dtype, H, Hk):
    B, T, d = 3, 37, 32
    _, q, k = norm_make(B, T, H, Hk, d, dtype, 3)
    kw = dict(inv_freq=freq(16))
    yq, yk = K.kata_qk_norm_rotate(q, k, **kw)
    gq, gk = torch.randn_like(yq), torch.randn_like(yk)
    dq, dk, _, _ = K.kata_qk_norm_rotate_backward(gq, gk, q, k, **kw)
    n = H + 2 * Hk
    for order in ((0, 1, 2), (0, 2, 1), (1, 0, 2), (2, 0, 1)):  # of batch, token, head in memory
        size = [(B, T, n)[x] for x in order] + [d]
        back = [order.index(x) for x in range(3)] + [3]
        buf = torch.full(size, 7.0, dtype=q.dtype, device="cuda")
        view = buf.permute(back)  # [B, T, n, d]
        K.kata_qk_norm_rotate_backward(gq, gk, q, k, dq=view[:, :, :H], dk=view[:, :, H:H + Hk], **kw)
        assert torch.equal(view[:, :, :H], dq) and torch.equal(view[:, :, H:H + Hk], dk), order
        assert bool((view[:, :, H + Hk:] == 7.0).all())
    # queries, keys and values head by head
    buf = torch.full((B, T, max(H, Hk), 3, d), 7.0, dtype=q.dtype, device="cuda")
    K.kata_qk_norm_rotate_backward(gq, gk, q, k, dq=buf[:, :, :H, 0], dk=buf[:, :, :Hk, 1], **kw)
    assert torch.equal(buf[:, :, :H, 0], dq) and torch.equal(buf[:, :, :Hk, 1], dk)
    assert bool((buf[:, :, :, 2] == 7.0).all()) and bool((buf[:, :, Hk:, 1] == 7.0).all())


def test_gradients_that_share_rows_are_refused():
    _, q, k = norm_make(2, 2, 1, 1, 64, "bf16", 4)
    g = torch.randn(2, 1, 2, 64, device="cuda").bfloat16()
    buf = torch.full((1024,), 7.0, dtype=torch.bfloat16, device="cuda")
    s = (192, 128, 64, 1)  # token 1 of sequence 0 of dk is token 0 of sequence 1 of dq
    with pytest.raises(K.KataError):
        K.kata_qk_norm_rotate_backward(g, g, q, k, dq=buf.as_strided(q.shape, s),
                                       dk=buf[64:].as_strided(k.shape, s))
    assert bool((buf == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk", [(50, 300), (3000, 40), (40, 1000)])
@pytest.mark.parametrize("where", ["query", "gradient"])
def test_gradients_of_padded_keys_are_zero_whatever_the_queries_hold(dtype, Tq, Tk, where):
    # one row that is not finite beside keys that end inside a tile: dk and dv of the
    # keys from the length on are zero all the same
    for d in (16, 64):
        q, k, v, g = make(3, 4, 2, Tq, Tk, d, dtype, seed=Tk + d)
        n = lens(Tk - 7, 0, Tk // 2 + 1)
        for bad in (float("nan"), float("inf")):
            (q if where == "query" else g)[:, 1, Tq // 2, 3] = bad
            _, y, den = forward(q, k, v, n)
            _, dk, dv = K.kata_cross_backward(g, q, k, v, y, den, key_lengths=n)
            for b in range(3):
                assert not dk[b, :, int(n[b]):].any() and not dv[b, :, int(n[b]):].any(), (d, bad, b)
                # key head 1 has none of the bad row
                assert bool(torch.isfinite(dk[b, 1]).all()) and bool(torch.isfinite(dv[b, 1]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Tq,Tk", [(2, 200, 300), (2, 1, 300), (8, 1, 5000), (2, 40, 100), (2, 3, 9000)])
def test_weights_below_the_normal_numbers_count_as_none(dtype, H, Tq, Tk):
    # s about 2^-72, l below 2^-126 though not 0 in fp32: zeros, as of a query without weight,
    # and nothing of that query in the keys' gradients
    q, k, v, g = make(2, H, 2, Tq, Tk, 64, dtype, seed=Tk)
    tiny, none = q.clone(), q.clone()
    tiny[:, :, Tq // 2] *= 2.0 ** -75
    none[:, :, Tq // 2] = 0
    for n in (None, lens(Tk, Tk // 2)):
        out, y, den = forward(tiny, k, v, n)
        assert not out[:, :, Tq // 2].any() and not y[:, :, Tq // 2].any()
        assert float(den[:, :, Tq // 2].max()) < 2.0 ** -126
        assert not K.kata_cross_forward(tiny, k, v, key_lengths=n)[:, :, Tq // 2].any()
        grads = K.kata_cross_backward(g, tiny, k, v, y, den, key_lengths=n)
        o0, y0, den0 = forward(none, k, v, n)
        assert torch.equal(out, o0)
        for a, b in zip(grads, K.kata_cross_backward(g, none, k, v, y0, den0, key_lengths=n)):
            assert torch.equal(a, b)


def test_a_pair_of_calls_in_an_autograd_function():
    # as the README has it
    class Cross(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, lengths):
            y = torch.empty(q.shape, dtype=torch.float32, device=q.device)
            den = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
            out = K.kata_cross_forward(q, k, v, key_lengths=lengths, y_out=y, den_out=den)
            ctx.save_for_backward(q, k, v, y, den, lengths)
            return out

        @staticmethod
        def backward(ctx, g):
            *saved, lengths = ctx.saved_tensors
            return (*K.kata_cross_backward(g.contiguous(), *saved, key_lengths=lengths), None)

    q, k, v, g = (t.requires_grad_() for t in make(2, 4, 2, 33, 70, 32, "f32", seed=21))
    assert not K.kata_cross_forward(q, k, v).requires_grad  # the call itself records nothing
    g = g.detach()
    for n in (None, lens(70, 11)):
        for up, loss in ((g, lambda t: (t * g).sum()), (torch.ones_like(g), lambda t: t.sum())):
            # the gradients of two uses add up
            got = torch.autograd.grad(loss(Cross.apply(q, k, v, n)) + loss(Cross.apply(q, k, v, n)), (q, k, v))
            ref = O.cross_grad(up, q.detach(), k.detach(), v.detach(), n)
            bounds = O.cross_bounds(q.detach(), k.detach(), v.detach(), torch.float32, n, dout=up)
            for a, r, b in zip(got, ref, bounds):
                assert O.worst(a / 2, r, b) <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,Tq,Tk", [(2, 2, 1, 300), (8, 2, 1, 5000), (6, 3, 11, 400), (4, 2, 33, 500), (4, 2, 300, 517)])
def test_a_bad_query_stays_in_its_row(dtype, H, Hk, Tq, Tk):
    # a query that is not finite, or overflows: the other rows of its tile, their gradients and
    # the other key heads' keep their bits
    q, k, v, g = make(2, H, Hk, Tq, Tk, 32, dtype, seed=Tk)
    n = lens(Tk, Tk // 2)
    a = forward(q, k, v, n)
    ga = K.kata_cross_backward(g, q, k, v, a[1], a[2], key_lengths=n)
    keep = torch.ones(2, H, Tq, dtype=torch.bool, device="cuda")
    keep[:, 0, Tq // 2] = False
    for value in (float("nan"), float("inf"), torch.finfo(q.dtype).max):
        bad = q.clone()
        bad[:, 0, Tq // 2, 1] = value
        b = forward(bad, k, v, n)
        gb = K.kata_cross_backward(g, bad, k, v, b[1], b[2], key_lengths=n)
        for x, y in zip(a + ga[:1], b + gb[:1]):
            assert torch.equal(x[keep], y[keep])
        for x, y in zip(ga[1:], gb[1:]):
            assert torch.equal(x[:, 1:], y[:, 1:])
