"""The head norm, the rotation and cross attention as a layer uses them: one after the
other beside the causal calls, step by step, on other streams, captured and
replayed, through the binding's short cut and without it."""
from __future__ import annotations

import pytest

from tests import layer_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import kernelized_linear_attention_fwd_b200 as K  # noqa: E402
from kernelized_linear_attention_fwd_b200 import binding  # noqa: E402
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


def layer(B, Tq, Tk, H, Hk, d, dtype, seed):
    """A decoder layer's inputs: its own fused projection, the queries of its cross
    attention, the encoder's fused keys and values."""
    g = gen(seed)

    def r(*s):
        return torch.randn(*s, device="cuda", generator=g).to(DT[dtype])

    return dict(own=r(B, Tq, 3 * H, d), q=r(B, Tq, H, d), enc=r(B, Tk, 2 * Hk, d),
                wq=1 + 0.2 * torch.randn(d, device="cuda", generator=g),
                wk=1 + 0.2 * torch.randn(d, device="cuda", generator=g),
                inv=(10000.0 ** (-torch.arange(d // 2, device="cuda").double() / (d // 2))).float())


def self_attention(x, H):
    q, k = K.kata_qk_norm_rotate(x["own"][:, :, :H], x["own"][:, :, H:2 * H], q_weight=x["wq"], k_weight=x["wk"],
                                 inv_freq=x["inv"])
    return q, k, x["own"][:, :, 2 * H:].transpose(1, 2).contiguous()


def cross_inputs(x, H, Hk):
    q, _ = K.kata_qk_norm_rotate(x["q"], q_weight=x["wq"])
    k, _ = K.kata_qk_norm_rotate(x["enc"][:, :, :Hk], q_weight=x["wk"])
    return q, k, x["enc"][:, :, Hk:].transpose(1, 2).contiguous()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_forward_and_gradient(dtype):
    B, Tq, Tk, H, Hk, d = 2, 150, 210, 4, 2, 64
    x = layer(B, Tq, Tk, H, Hk, d, dtype, 1)
    n = torch.tensor([Tk, 77], dtype=torch.int32, device="cuda")
    # self attention of normed, rotated queries and keys
    q, k, v = self_attention(x, H)
    out = K.kata_chunked_forward(q, k, v)
    s = (q.double() @ k.double().transpose(-1, -2)).tril() ** 2
    ref = s @ v.double() / s.sum(-1, keepdim=True)
    tol = 2e-2 if dtype == "bf16" else 1e-4
    assert float(((out.double() - ref).abs().amax(-1) / ref.abs().amax(-1)).max()) <= tol
    # cross attention of normed queries and keys, its gradient, and the norms' gradients
    q, k, v = cross_inputs(x, H, Hk)
    y = torch.empty(q.shape, device="cuda")
    den = torch.empty(q.shape[:3], device="cuda")
    out = K.kata_cross_forward(q, k, v, key_lengths=n, y_out=y, den_out=den)
    ref, _ = O.cross(q, k, v, n)
    assert O.worst(out, ref, O.cross_bounds(q, k, v, q.dtype, n)[0]) <= 1
    g = torch.randn(out.shape, device="cuda", generator=gen(2)).to(out.dtype)
    grads = K.kata_cross_backward(g, q, k, v, y, den, key_lengths=n)
    for a, r, b in zip(grads, O.cross_grad(g, q, k, v, n), O.cross_bounds(q, k, v, q.dtype, n, dout=g)):
        assert O.worst(a, r, b) <= 1
    none = O.angles(None, None, B, Tq, "cuda")
    dx, _, dw, _ = K.kata_qk_norm_rotate_backward(grads[0], None, x["q"], q_weight=x["wq"])
    rx, rw = O.norm_rotate_grad(grads[0], x["q"], x["wq"], none, 1e-6, False)
    bx, bw = O.norm_grad_bounds(rx, grads[0], x["q"], x["wq"], dx.dtype, 1e-6, False, 0)
    assert O.worst(dx, rx, bx) <= 1 and O.worst(dw, rw, bw) <= 1


def test_whole_chain_gradient_against_differences():
    # fp32: the gradient of sum(g * cross(norm(q), norm(k), v)) by its three calls
    x = layer(1, 5, 7, 2, 1, 16, "f32", 3)
    g = torch.randn(1, 2, 5, 16, device="cuda", generator=gen(4))
    q, k, v = cross_inputs(x, 2, 1)
    y, den = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:3], device="cuda")
    K.kata_cross_forward(q, k, v, y_out=y, den_out=den)
    dq, dk, _ = K.kata_cross_backward(g, q, k, v, y, den)
    dxq = K.kata_qk_norm_rotate_backward(dq, None, x["q"], q_weight=x["wq"])[0]
    dxk = K.kata_qk_norm_rotate_backward(dk, None, x["enc"][:, :, :1], q_weight=x["wk"])[0]
    none = O.angles(None, None, 1, 7, "cuda")

    def f(xq, xk):
        qq = O.norm_rotate(xq, x["wq"], none[:, :, :5], 1e-6, False)
        kk = O.norm_rotate(xk, x["wk"], none, 1e-6, False)
        return float((O.cross(qq, kk, v)[0] * g.double()).sum())

    h = 1e-6
    for seed in range(3):
        e = torch.randn(x["q"].shape, device="cuda", generator=gen(seed)).double()
        u = torch.randn(1, 7, 1, 16, device="cuda", generator=gen(seed + 5)).double()
        xk = x["enc"][:, :, :1].double()
        num = (f(x["q"].double() + h * e, xk + h * u) - f(x["q"].double() - h * e, xk - h * u)) / (2 * h)
        ana = float((dxq.double() * e).sum() + (dxk.double() * u).sum())
        scale = float((dxq.double() * e).abs().sum() + (dxk.double() * u).abs().sum())
        # fp32 through three calls: sums of at most 64 terms each, 1000 U of the magnitudes
        assert abs(num - ana) <= 1000 * O.U * scale + 1e-7 * scale


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_steps_give_the_rows_of_the_whole(dtype):
    B, T, Tk, H, Hk, d = 3, 6, 500, 4, 2, 32
    x = layer(B, T, Tk, H, Hk, d, dtype, 7)
    n = torch.tensor([Tk, 130, 0], dtype=torch.int32, device="cuda")
    pos = torch.tensor([[100], [5], [70000]], device="cuda") + torch.arange(T, device="cuda")
    whole, wk = K.kata_qk_norm_rotate(x["own"][:, :, :H], x["own"][:, :, H:2 * H], inv_freq=x["inv"], positions=pos)
    k, _ = K.kata_qk_norm_rotate(x["enc"][:, :, :Hk])
    v = x["enc"][:, :, Hk:].transpose(1, 2).contiguous()
    out = K.kata_cross_forward(whole, k, v, key_lengths=n)
    ref, _ = O.cross(whole, k, v, n)
    for t in range(T):
        q1, k1 = K.kata_qk_norm_rotate(x["own"][:, t:t + 1, :H], x["own"][:, t:t + 1, H:2 * H], inv_freq=x["inv"],
                                       positions=pos[:, t:t + 1])
        assert torch.equal(q1[:, :, 0], whole[:, :, t]) and torch.equal(k1[:, :, 0], wk[:, :, t])
        o1 = K.kata_cross_forward(q1, k, v, key_lengths=n)
        b = O.cross_bounds(q1, k, v, q1.dtype, n)[0]
        assert O.worst(o1, ref[:, :, t:t + 1], b) <= 1
        assert O.worst(o1, out[:, :, t:t + 1].double(), 2 * b) <= 1


def everything(x, H, Hk, n, g, stream=None):
    """Every call once; all outputs."""
    q, k = K.kata_qk_norm_rotate(x["q"], x["enc"][:, :, :Hk].contiguous()[:, :x["q"].shape[1]], q_weight=x["wq"],
                                 k_weight=x["wk"], inv_freq=x["inv"], stream=stream)
    gk = k * 1
    a = K.kata_qk_norm_rotate_backward(q, gk, x["q"], x["enc"][:, :x["q"].shape[1], :Hk], q_weight=x["wq"],
                                       k_weight=x["wk"], inv_freq=x["inv"], stream=stream)
    ke = x["k"]
    y, den = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:3], device="cuda")
    out = K.kata_cross_forward(q, ke, x["v"], key_lengths=n, y_out=y, den_out=den, stream=stream)
    b = K.kata_cross_backward(g, q, ke, x["v"], y, den, key_lengths=n, stream=stream)
    return (q, k, out, y, den) + a + b


def prepared(B, Tq, Tk, H, Hk, d, dtype, seed):
    x = layer(B, Tq, Tk, H, Hk, d, dtype, seed)
    x["k"] = x["enc"][:, :, :Hk].transpose(1, 2).contiguous()
    x["v"] = x["enc"][:, :, Hk:].transpose(1, 2).contiguous()
    n = torch.randint(0, Tk + 1, (B,), device="cuda", generator=gen(seed)).int()
    g = torch.randn(B, H, Tq, d, device="cuda", generator=gen(seed + 1)).to(DT[dtype])
    return x, n, g


SHAPES = [(2, 70, 3000, 4, 2, 64, "bf16"), (2, 3, 5000, 2, 2, 32, "bf16"), (2, 40, 700, 4, 2, 32, "f32")]


@pytest.mark.parametrize("shape", SHAPES)
def test_short_cut_and_python_path_agree(shape, monkeypatch):
    if binding._calls is None:
        pytest.skip("built without the short cut")
    x, n, g = prepared(*shape, 11)
    a = everything(x, shape[3], shape[4], n, g)
    monkeypatch.setattr(binding, "_calls", None)
    b = everything(x, shape[3], shape[4], n, g)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


@pytest.mark.parametrize("shape", SHAPES)
def test_other_streams(shape):
    x, n, g = prepared(*shape, 13)
    ref = everything(x, shape[3], shape[4], n, g)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):  # two streams at a time, each with its own buffers
        with torch.cuda.stream(s1):
            a = everything(x, shape[3], shape[4], n, g)
        with torch.cuda.stream(s2):
            b = everything(x, shape[3], shape[4], n, g, stream=s2)
        got += [a, b]
    torch.cuda.synchronize()
    for a in got:
        for u, v in zip(ref, a):
            assert torch.equal(u, v)


@pytest.mark.parametrize("shape", SHAPES)
def test_captured_and_replayed(shape):
    x, n, g = prepared(*shape, 17)
    everything(x, shape[3], shape[4], n, g)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs, each with the memory of its own capture
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = everything(x, shape[3], shape[4], n, g)
        graphs.append((gr, out))
    x2, n2, g2 = prepared(*shape, 18)
    want = everything(x2, shape[3], shape[4], n2, g2)
    for key in ("q", "enc", "k", "v"):
        x[key].copy_(x2[key])
    for key in ("wq", "wk", "inv"):
        x[key].copy_(x2[key])
    n.copy_(n2)
    g.copy_(g2)
    for gr, _ in graphs * 2:
        gr.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        for u, v in zip(want, out):
            assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk", [(1, 9000), (3, 300), (130, 700), (64, 64)])
def test_nothing_around_the_outputs_is_written(dtype, Tq, Tk):
    B, H, Hk, d = 2, 4, 2, 32
    x, n, g = prepared(B, Tq, Tk, H, Hk, d, dtype, 19)
    q = torch.randn(B, H, Tq, d, device="cuda", generator=gen(1)).to(DT[dtype])

    def guarded(shape, dt):
        size = 1
        for s in shape:
            size *= s
        raw = torch.full((size + 512,), 7.0, dtype=dt, device="cuda")
        return raw, raw[256:256 + size].view(shape)

    code = 1 if dtype == "bf16" else 0
    raws, bufs = zip(*[guarded(s, dt) for s, dt in [
        (q.shape, q.dtype), (q.shape, torch.float32), (q.shape[:3], torch.float32), (q.shape, q.dtype),
        (x["k"].shape, q.dtype), (x["k"].shape, q.dtype)]])
    out, y, den, dq, dk, dv = bufs
    wf = torch.full((K.kata_cross_forward_workspace_bytes(B, H, Hk, Tq, Tk, d, code) + 1024,), 9, dtype=torch.uint8,
                    device="cuda")
    wb = torch.full((K.kata_cross_backward_workspace_bytes(B, H, Hk, Tq, Tk, d, code) + 1024,), 9, dtype=torch.uint8,
                    device="cuda")
    K.kata_cross_forward(q, x["k"], x["v"], key_lengths=n, out=out, y_out=y, den_out=den, workspace=wf[:-1024])
    K.kata_cross_backward(g, q, x["k"], x["v"], y, den, key_lengths=n, dq=dq, dk=dk, dv=dv, workspace=wb[:-1024])
    for raw in raws:
        assert bool((raw[:256] == 7).all()) and bool((raw[-256:] == 7).all())
    assert bool((wf[-1024:] == 9).all()) and bool((wb[-1024:] == 9).all())
    ref, _ = O.cross(q, x["k"], x["v"], n)
    assert O.worst(out, ref, O.cross_bounds(q, x["k"], x["v"], q.dtype, n)[0]) <= 1


def test_refused_calls_leave_the_library_usable():
    x, n, g = prepared(2, 20, 30, 4, 2, 32, "bf16", 23)
    q = torch.randn(2, 4, 20, 32, device="cuda").bfloat16()
    k, v = x["k"], x["v"]
    ok = K.kata_cross_forward(q, k, v, key_lengths=n)
    bad = [
        lambda: K.kata_cross_forward(q.float(), k, v),
        lambda: K.kata_cross_forward(q.half(), k.half(), v.half()),
        lambda: K.kata_cross_forward(q[:, :, ::2], k, v),
        lambda: K.kata_cross_forward(q, k[:1], v),
        lambda: K.kata_cross_forward(q, k, v[:, :, :-1]),
        lambda: K.kata_cross_forward(q[:, :3].contiguous(), k, v),
        lambda: K.kata_cross_forward(q, k, v, key_lengths=n.long()),
        lambda: K.kata_cross_forward(q, k, v, key_lengths=n[:1]),
        lambda: K.kata_cross_forward(q, k, v, key_lengths=n.cpu()),
        lambda: K.kata_cross_forward(q, k.cpu(), v),
        lambda: K.kata_cross_forward(q, k, v, out=q),
        lambda: K.kata_cross_forward(q, k, v, y_out=torch.empty_like(q)),
        lambda: K.kata_cross_forward(q[:, :, :0], k, v),
        lambda: K.kata_cross_forward(q, k[:, :, :0], v[:, :, :0]),
        lambda: K.kata_cross_backward(g, q, k, v, None, None),
        lambda: K.kata_cross_backward(None, q, k, v, q.float(), q[..., 0].float().contiguous()),
        lambda: K.kata_cross_backward(g, q, k, v, q.float(), q[..., 0].float().contiguous(),
                                      workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: K.kata_qk_norm_rotate(x["q"].half()),
        lambda: K.kata_qk_norm_rotate(x["q"], x["enc"][:, :-1, :2]),
        lambda: K.kata_qk_norm_rotate(x["q"][..., ::2]),
        lambda: K.kata_qk_norm_rotate(x["q"], k_weight=x["wk"]),
        lambda: K.kata_qk_norm_rotate(x["q"], q_weight=x["wq"].bfloat16()),
        lambda: K.kata_qk_norm_rotate(x["q"], inv_freq=x["inv"].double()),
        lambda: K.kata_qk_norm_rotate(x["q"], inv_freq=torch.ones(17, device="cuda")),
        lambda: K.kata_qk_norm_rotate(x["q"], inv_freq=torch.ones(6, device="cuda")),
        lambda: K.kata_qk_norm_rotate(x["q"], inv_freq=x["inv"], positions=torch.zeros(20, device="cuda")),
        lambda: K.kata_qk_norm_rotate(x["q"], inv_freq=x["inv"],
                                      positions=torch.zeros(19, dtype=torch.int64, device="cuda")),
        lambda: K.kata_qk_norm_rotate(x["q"], eps=0.0),
        lambda: K.kata_qk_norm_rotate(x["q"], q_out=x["q"]),
        lambda: K.kata_qk_norm_rotate(x["q"][:, :, :0]),
        lambda: K.kata_qk_norm_rotate_backward(None, None, x["q"]),
        lambda: K.kata_qk_norm_rotate_backward(q, q, x["q"]),
        lambda: K.kata_qk_norm_rotate_backward(q, None, x["q"], dq=x["q"]),
        lambda: K.kata_qk_norm_rotate_backward(q, None, x["q"], dq=x["q"].new_empty(1, 20, 4, 32).expand(2, -1, -1, -1)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(K.KataError):
            f()
            pytest.fail(f"call {i} was taken")
    assert torch.equal(ok, K.kata_cross_forward(q, k, v, key_lengths=n))


@pytest.mark.parametrize("Tq", [1, 130])
def test_keys_past_2_to_31_elements(Tq):
    # 33 key heads of 2^20 keys: the last head lies past 2^31 elements
    B, H, Tk, d = 1, 33, 2 ** 20, 64
    k = torch.zeros(B, H, Tk, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[0, -1] = torch.randn(Tk, d, device="cuda", generator=gen(1)).bfloat16()
    v[0, -1] = torch.randn(Tk, d, device="cuda", generator=gen(2)).bfloat16()
    q = torch.randn(B, H, Tq, d, device="cuda", generator=gen(3)).bfloat16()
    y = torch.empty(q.shape, device="cuda")
    den = torch.empty(q.shape[:3], device="cuda")
    K.kata_cross_forward(q, k, v, y_out=y, den_out=den)
    assert not y[0, :-1].any()
    rows = slice(0, min(Tq, 4))
    s = (q[0, -1, rows].double() @ k[0, -1].double().T) ** 2
    ref = s @ v[0, -1].double() / s.sum(-1, keepdim=True)
    # random signs: 2^-8 of each weight's share of v - y, six standard deviations of their sum,
    # and 2^-12 of it for the fp32 sums in the tensor cores (2^16 additions of 2^-24, truncated)
    p = s / s.sum(-1, keepdim=True)
    tol = 6 * 2.0 ** -8 * ((p ** 2) @ (v[0, -1].double() ** 2)).sqrt() + 2.0 ** -8 * ref.abs() + \
        2.0 ** -12 * (p @ v[0, -1].double().abs())
    assert float(((y[0, -1, rows].double() - ref).abs() / tol).max()) <= 1
    if Tq == 1:
        g = torch.randn(q.shape, device="cuda", generator=gen(4)).bfloat16()
        dq, dk, dv = K.kata_cross_backward(g, q, k, v, y, den)
        rv = p.T @ g[0, -1].double()
        assert float((dv[0, -1].double() - rv).abs().max()) <= 2.0 ** -6 * float(rv.abs().max())
        assert not dk[0, :-1].any() and not dv[0, :-1].any()
