"""The binding's two ways into the layer calls, the short cut and the Python path, give the
same bits for what they take and the same status for what they refuse."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import kernelized_linear_attention_fwd_b200 as K  # noqa: E402
from kernelized_linear_attention_fwd_b200 import binding  # noqa: E402
from kernelized_linear_attention_fwd_b200.csrc import build as kbuild  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    K.load_library()
    yield
    assert K.kata_get_device_status() == 0


class Sub(torch.Tensor):
    pass


def outcome(f):
    """What a call gives: its outputs, or the status and the type of its refusal."""
    try:
        r = f()
    except K.KataError as e:
        return "refused", e.status
    return tuple(r) if isinstance(r, tuple) else (r,)


def refused(a):
    return isinstance(a[0], str)


def same(a, b):
    if refused(a) or refused(b):
        return refused(a) and refused(b) and a == b
    return len(a) == len(b) and all(
        x is None and y is None or x is not None and y is not None and torch.equal(x, y)
        and x.stride() == y.stride() and x.dtype == y.dtype for x, y in zip(a, b))


def cases():
    g = torch.Generator(device="cuda").manual_seed(1)

    def r(*s, dt=torch.bfloat16):
        return torch.randn(*s, device="cuda", generator=g).to(dt)

    B, T, H, Hk, d = 2, 20, 4, 2, 32
    p = r(B, T, H + 2 * Hk, d)
    q, k, k1 = p[:, :, :H], p[:, :, H:H + Hk], p[:, :, H:H + 1]
    w, inv = r(d, dt=torch.float32), torch.rand(16, device="cuda", generator=g)
    pos = torch.randint(0, 999, (B, T), device="cuda", generator=g)
    gq, gk, gk1 = r(B, H, T, d), r(B, Hk, T, d), r(B, 1, T, d)
    f32 = torch.float32
    N, D = K.kata_qk_norm_rotate, K.kata_qk_norm_rotate_backward
    need = K.kata_qk_norm_rotate_backward_workspace_bytes(B, T, H, Hk, d)

    def new(*s, dt=torch.bfloat16):
        return torch.full(s, 3.0, dtype=dt, device="cuda")

    norm = [
        lambda: N(q), lambda: N(q, k), lambda: N(q, k1), lambda: N(q.float(), k.float(), w, w, inv, pos),
        lambda: N(q, k, w, w, inv, pos, 1e-3, True), lambda: N(q, k, None, w, inv[:5], None, 1, 1),
        lambda: N(q, None, w, None, inv[:0], pos[0]), lambda: N(q, inv_freq=inv, positions=pos[:, :1].expand(B, T)),
        lambda: N(q[:1], inv_freq=inv, positions=pos[:1]), lambda: N(q[:, :1], inv_freq=inv, positions=pos[:, 3:4]),
        lambda: N(q, inv_freq=inv, positions=pos[:1].expand(B, T)), lambda: N(q[:1].expand(3, -1, -1, -1)),
        lambda: N(q.transpose(1, 2).contiguous().transpose(1, 2), k), lambda: N(q, q_out=new(B, H, T, d)),
        lambda: N(q, k, k_out=new(B, Hk, T, d)), lambda: N(torch.nn.Parameter(q.detach().clone())),
        lambda: N(q.as_subclass(Sub), k), lambda: N(q, q_weight=torch.nn.Parameter(w)),
        lambda: N(q, k_out=new(B, Hk, T, d)), lambda: N(q, k, q_out=new(B, H, T, d, dt=f32)),
        lambda: N(q, k, k_out=new(B, Hk, T, d)[:, :, ::2]), lambda: N(q, k.float()), lambda: N(q, k[:1]),
        lambda: N(q, k[..., :16]), lambda: N(q[..., 1:17]), lambda: N(q[..., :24]), lambda: N(q[0]),
        lambda: N(q, w[:16]), lambda: N(q, w.double()), lambda: N(q, w[None]), lambda: N(q, None, None, w),
        lambda: N(q, inv_freq=inv[None]), lambda: N(q, inv_freq=inv[::2]), lambda: N(q, inv_freq=inv.half()),
        lambda: N(q, inv_freq=inv[:3]), lambda: N(q, inv_freq=inv.repeat(2)), lambda: N(q, inv_freq=inv, positions=pos.int()),
        lambda: N(q, inv_freq=inv, positions=pos[:, :-1]), lambda: N(q, inv_freq=inv, positions=pos.T.contiguous().T),
        lambda: N(q, inv_freq=inv, positions=pos.cpu()), lambda: N(q, inv_freq=inv.cpu()), lambda: N(q, eps=0),
        lambda: N(q, eps=-1.0), lambda: N(q, eps=float("nan")), lambda: N(q, eps=1e60), lambda: N(q, eps=1e-60),
        lambda: N(q[:0]), lambda: N(q[:, :0]), lambda: N(q, k[:, :, :0]), lambda: N(q, k, k_out=q[:, :, :Hk]),
        lambda: N(q.half(), k.half()), lambda: N(q.to(torch.float8_e4m3fn)), lambda: N(q, q_out=q),
    ]
    grad = [
        lambda: D(gq, None, q), lambda: D(gq, gk, q, k), lambda: D(gq, gk, q, k, w, w, inv, pos, 1e-3, True),
        lambda: D(gq.float(), gk.float(), q.float(), k.float(), w, None, inv), lambda: D(gq, gk1, q, k1, None, w),
        lambda: D(gq, gk, q, k, dq=new(B, H, T, d).transpose(1, 2)),
        lambda: D(gq, gk, q, k, dk=new(B, T, Hk + 1, d)[:, :, 1:]),
        lambda: D(gq, gk, q, k, dq_weight=new(d, dt=f32), dk_weight=new(d, dt=f32)),
        lambda: D(gq, gk, q, k, workspace=torch.empty(need, dtype=torch.uint8, device="cuda")),
        lambda: D(gq, gk, q, k, workspace=torch.empty(need // 4, dtype=f32, device="cuda")),
        lambda: D(gq, gk, q, k, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda")),
        lambda: D(gq, gk, q, k, workspace=torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:]),
        lambda: D(gq, gk, q, k, workspace=torch.empty(need, dtype=torch.uint8)),
        lambda: D(gq, gk, q, k, workspace=torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]),
        lambda: D(None, gk, q, k), lambda: D(gq, None, q, k), lambda: D(gq, gk, q), lambda: D(gq.transpose(1, 2), None, q),
        lambda: D(gq.float(), None, q), lambda: D(gq, gk, q, k, dk=new(B, T, Hk, d, dt=f32)),
        lambda: D(gq, None, q, dk=new(B, T, Hk, d)), lambda: D(gq, None, q, dk_weight=new(d, dt=f32)),
        lambda: D(gq, gk, q, k, dq=new(B, T, H + 1, d)), lambda: D(gq, gk, q, k, dq=new(B, T, H, 2 * d)[..., ::2]),
        lambda: D(gq, gk, q, k, dq_weight=new(d)), lambda: D(gq, gk, q, k, dq=q), lambda: D(gq, gk, q, k, dk_weight=w[:16]),
    ]
    c, kk, v = r(B, H, T, d), r(B, Hk, 50, d), r(B, Hk, 50, d)
    n = torch.tensor([50, 17], dtype=torch.int32, device="cuda")
    F, X = K.kata_cross_forward, K.kata_cross_backward
    y, den = torch.empty(c.shape, device="cuda"), torch.empty(c.shape[:3], device="cuda")
    F(c, kk, v, n, y_out=y, den_out=den)
    go, long = r(B, H, T, d), r(B, Hk, 9000, d)
    need_f = K.kata_cross_forward_workspace_bytes(B, H, Hk, 1, 9000, d, binding.KATA_BF16)
    one = c[:, :, :1].contiguous()

    def bytes_(x):
        return torch.empty(x, dtype=torch.uint8, device="cuda")

    cross = [
        lambda: F(c, kk, v), lambda: F(c, kk, v, n), lambda: F(c.float(), kk.float(), v.float(), n),
        lambda: F(c, kk, v, n, new(*c.shape)), lambda: F(c, kk, v, n, None, new(*c.shape, dt=f32), new(*c.shape[:3], dt=f32)),
        lambda: F(one, long, long), lambda: F(one, long, long, workspace=bytes_(need_f)),
        lambda: F(one, long, long, workspace=bytes_(need_f - 1)), lambda: F(one, long, long, workspace=bytes_(need_f + 8)[8:]),
        lambda: F(c.as_subclass(Sub), kk, v), lambda: F(torch.nn.Parameter(c), kk, v),
        lambda: F(c, kk, None), lambda: F(c, kk[0], v), lambda: F(c, kk, v[:, :1]), lambda: F(c[..., :24].contiguous(), kk, v),
        lambda: F(c, kk, v.float()), lambda: F(c, kk, v, n.long()), lambda: F(c, kk, v, n.cpu()), lambda: F(c, kk, v, n[None]),
        lambda: F(c, kk, v, n, new(*c.shape, dt=f32)), lambda: F(c, kk, v, n, c), lambda: F(c, kk, v, y_out=new(*c.shape)),
        lambda: F(c, kk, v, den_out=new(B, H, T, 1, dt=f32)), lambda: F(c[:, :3].contiguous(), kk, v), lambda: F(c[:0], kk[:0], v[:0]),
        lambda: F(c.transpose(1, 2).contiguous().transpose(1, 2), kk, v), lambda: F(c.half(), kk.half(), v.half()),
        lambda: X(go, c, kk, v, y, den, n), lambda: X(go, c, kk, v, y, den, n, new(*c.shape), new(*kk.shape), new(*kk.shape)),
        lambda: X(go, c, kk, v, y, den, n, workspace=bytes_(1 << 24)), lambda: X(go, c, kk, v, y, den, n, workspace=bytes_(64)),
        lambda: X(go.float(), c, kk, v, y, den, n), lambda: X(go, c, kk, v, y.bfloat16(), den, n),
        lambda: X(go, c, kk, v, y, den[..., None], n), lambda: X(go, c, kk, v, y, None, n), lambda: X(None, c, kk, v, y, den, n),
        lambda: X(go, c, kk, v, y, den, n, dq=go), lambda: X(go, c, kk, v, y, den, n, dk=new(*kk.shape, dt=f32)),
        lambda: X(go, c, kk, v, y, den, n, dv=new(B, Hk, 49, d)),
    ]
    return norm + grad + cross


def test_both_ways_agree_on_every_call(monkeypatch):
    if binding._calls is None:
        pytest.skip("built without the short cut")
    got, calls = [], cases()
    for f in calls:
        got.append(outcome(f))
    monkeypatch.setattr(binding, "_calls", None)
    taken = 0
    for i, (f, a) in enumerate(zip(calls, got)):
        b = outcome(f)
        assert same(a, b), (i, a if refused(a) else "taken", b if refused(b) else "taken")
        taken += not refused(a)
    assert 35 < taken < len(calls) - 50
