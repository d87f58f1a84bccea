"""Operators around the KATA attention that are measured case by case.

Four operators of a layer that attends to another sequence:

  norm        kata_qk_norm_rotate: per-head RMS norm of queries and keys and the
              rotation by position, token-major projections in, head-major out
  norm_grad   the same and its gradient (a training step through it)
  cross       kata_cross_forward: y_t = sum_s (q_t.k_s)^2 v_s / sum_s (q_t.k_s)^2
              over the first key_lengths[b] of Tk keys (0 where the sum is 0)
  cross_grad  the same and its gradient

`run` computes them in plain torch operations in 32 bits (angles in 64) when
`own` is false, and through the package's entry points when it is true.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6


def listed():
    return [
        # one decode step of 64 sequences, 16 heads: every sequence at its own far position
        dict(name="norm_decode_b64", op="norm", B=64, T=1, H=16, Hk=16, d=64, rot=64,
             inter=False, dtype="bf16"),
        # prefill of the 340M-parameter shape, the projections one fused matrix
        dict(name="norm_prefill_16k", op="norm", B=4, T=16384, H=16, Hk=16, d=64, rot=64,
             inter=False, dtype="bf16"),
        # odd length, fp32, shared key heads, partial rotation of neighbouring pairs
        dict(name="norm_odd_f32", op="norm", B=2, T=4093, H=12, Hk=3, d=32, rot=24,
             inter=True, dtype="f32"),
        # a training step on a long sequence
        dict(name="norm_grad_long", op="norm_grad", B=1, T=32768, H=16, Hk=4, d=64, rot=64,
             inter=False, dtype="bf16"),
        # a small ragged fp32 training step
        dict(name="norm_grad_small_f32", op="norm_grad", B=3, T=517, H=4, Hk=4, d=16, rot=16,
             inter=False, dtype="f32"),
        # one decoder token of 64 sequences against padded encoder states
        dict(name="cross_decode_b64", op="cross", B=64, H=16, Hk=16, Tq=1, Tk=1501, d=64,
             ragged=True, dtype="bf16"),
        # one token, shared key heads, one very long memory
        dict(name="cross_decode_long", op="cross", B=1, H=16, Hk=2, Tq=1, Tk=131072, d=64,
             ragged=False, dtype="bf16"),
        # a whole decoder sequence against a long encoder sequence
        dict(name="cross_prefill", op="cross", B=1, H=8, Hk=8, Tq=8192, Tk=16384, d=64,
             ragged=False, dtype="bf16"),
        # small fp32 heads of odd lengths
        dict(name="cross_small_f32", op="cross", B=2, H=4, Hk=4, Tq=77, Tk=333, d=32,
             ragged=True, dtype="f32"),
        # a training step, decoder shorter than the padded encoder
        dict(name="cross_grad_mid", op="cross_grad", B=4, H=16, Hk=16, Tq=2048, Tk=4096, d=64,
             ragged=True, dtype="bf16"),
        # a training step with shared key heads and odd lengths
        dict(name="cross_grad_shared", op="cross_grad", B=2, H=8, Hk=2, Tq=1021, Tk=1999, d=32,
             ragged=False, dtype="bf16"),
        # a small fp32 training step
        dict(name="cross_grad_f32", op="cross_grad", B=2, H=4, Hk=2, Tq=301, Tk=517, d=64,
             ragged=True, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "cross", "cross_grad"])
    d = rng.choice([16, 32, 64, 64])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hk = rng.choice([1, 2, 3, 4, 8])
    H = Hk * rng.choice([1, 1, 2, 4])
    if op in ("norm", "norm_grad"):
        B = rng.choice([1, 2, 3, 8, 37])
        # at most the prefill's 4 * 16384 * 32 rows of 64 bf16 (norm), the long step's (grad)
        rows = 2 ** 20 if op == "norm" else 2 ** 18
        T = _log_int(rng, 1, max(1, rows // (B * (H + Hk))))
        inter = rng.random() < 0.5
        rot = rng.choice([8 * i for i in range(1, d // 8 + 1)])
        return dict(op=op, B=B, T=T, H=H, Hk=Hk, d=d, rot=rot, inter=inter, dtype=dtype)
    B = rng.choice([1, 2, 3, 7])
    # score entries of all heads: well below the prefill's 2^30 and the step's 2^29,
    # fewer in fp32
    area = (2 ** 28 if dtype == "bf16" else 2 ** 25) // (B * H)
    Tq = 1 if (op == "cross" and rng.random() < 0.3) else _log_int(rng, 1, 4096)
    Tk = _log_int(rng, 1, max(1, min(65536, area // Tq)))
    return dict(op=op, B=B, H=H, Hk=Hk, Tq=Tq, Tk=Tk, d=d, ragged=rng.random() < 0.5, dtype=dtype)


def _lengths(case):
    """Keys each sequence may attend to: full, or between about 3/8 and all of
    the keys, the last sequence of three or more having none."""
    B, Tk = case["B"], case["Tk"]
    if not case["ragged"]:
        return [Tk] * B
    n = [max(1, Tk - (5 * b * Tk) // (8 * B)) for b in range(B)]
    if B >= 3:
        n[-1] = 0
    return n


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    g = _gen(seed)
    dt = _DT[case["dtype"]]
    dev = "cuda"

    def randn(*shape):
        return torch.randn(*shape, device=dev, generator=g)

    B, H, Hk, d = case["B"], case["H"], case["Hk"], case["d"]
    st = dict(case=case)
    if case["op"] in ("norm", "norm_grad"):
        T, n = case["T"], case["rot"] // 2
        # one fused projection [B, T, (H + 2 Hk) d]: queries, keys, values side by side
        proj = randn(B, T, H + 2 * Hk, d)
        proj *= torch.exp(0.5 * randn(B, T, H + 2 * Hk, 1))
        st["proj"] = proj.to(dt)
        st["q"] = st["proj"][:, :, :H]
        st["k"] = st["proj"][:, :, H:H + Hk]
        st["wq"] = 1.0 + 0.2 * randn(d)
        st["wk"] = 1.0 + 0.2 * randn(d)
        st["inv_freq"] = (10000.0 ** (-torch.arange(n, device=dev, dtype=torch.float64) / n)).float()
        first = torch.randint(0, 131072, (B, 1), device=dev, generator=g)
        st["pos"] = first + torch.arange(T, device=dev)[None, :]
        if case["op"] == "norm_grad":
            st["gq"] = randn(B, H, T, d).to(dt)
            st["gk"] = randn(B, Hk, T, d).to(dt)
        return st
    Tq, Tk = case["Tq"], case["Tk"]

    def unit_rms(x):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)

    st["q"] = unit_rms(randn(B, H, Tq, d)).to(dt)
    st["k"] = unit_rms(randn(B, Hk, Tk, d)).to(dt)
    st["v"] = randn(B, Hk, Tk, d).to(dt)
    st["len"] = (torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
                 if case["ragged"] else None)
    if case["op"] == "cross_grad":
        st["g"] = randn(B, H, Tq, d).to(dt)
    return st


# ----------------------------------------------------------------- plain form

def _angles(st):
    a = st["pos"].double()[..., None] * st["inv_freq"].double()
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin, inter, sign):
    """Rotation of the first 2 n coordinates of x [B, H, T, d] by the angles [B, T, n]."""
    n = cos.shape[-1]
    c, s = cos[:, None], sign * sin[:, None]
    if inter:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
    else:
        a, b = x[..., :n], x[..., n:2 * n]
    ra, rb = a * c - b * s, a * s + b * c
    out = x.clone()
    if inter:
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = ra, rb
    else:
        out[..., :n], out[..., n:2 * n] = ra, rb
    return out


def _plain_norm(x, w, cos, sin, inter):
    f = x.float().transpose(1, 2)
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + _EPS)
    return _rotate(f * r * w, cos, sin, inter, 1.0).to(x.dtype)


def _plain_norm_grad(gy, x, w, cos, sin, inter):
    f = x.float().transpose(1, 2)
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + _EPS)
    g = _rotate(gy.float(), cos, sin, inter, -1.0)
    u = f * r
    dw = (g * u).sum((0, 1, 2))
    gw = g * w
    dx = r * (gw - u * (gw * u).mean(-1, keepdim=True))
    return dx.transpose(1, 2).to(x.dtype), dw


def _slabs(B, Hk, per_head):
    """Pieces (b, first key head, last key head + 1) of at most 2^29 score entries."""
    step = max(1, min(Hk, 2 ** 29 // max(1, per_head)))
    return [(b, h, min(Hk, h + step)) for b in range(B) for h in range(0, Hk, step)]


def _plain_cross(st, grad):
    case = st["case"]
    B, H, Hk, Tq, Tk, d = (case[x] for x in ("B", "H", "Hk", "Tq", "Tk", "d"))
    q, k, v, n = st["q"], st["k"], st["v"], st["len"]
    R = (H // Hk) * Tq
    qf = q.reshape(B, Hk, R, d)
    mask = None
    if n is not None:
        mask = torch.arange(Tk, device=q.device)[None, :] < n[:, None]
    out = torch.empty_like(qf)
    if B * Hk * R * Tk <= 2 ** 29:  # all heads at once, else piece by piece
        parts = [(slice(None), slice(None))]
    else:
        parts = [(slice(b, b + 1), slice(h0, h1)) for b, h0, h1 in _slabs(B, Hk, R * Tk)]
    if grad:
        gf = st["g"].reshape(B, Hk, R, d)
        dq, dk, dv = torch.empty_like(qf), torch.empty_like(k), torch.empty_like(v)
    for b, h in parts:
        qs, ks, vs = qf[b, h].float(), k[b, h].float(), v[b, h].float()
        s = qs @ ks.transpose(-1, -2)
        if mask is not None:
            s = s * mask[b][:, None, None, :]
        w = s * s
        den = w.sum(-1, keepdim=True)
        inv = torch.where(den > 0, 1.0 / den, torch.zeros_like(den))
        p = w * inv
        y = p @ vs
        out[b, h] = y.to(q.dtype)
        if grad:
            gs = gf[b, h].float()
            dv[b, h] = (p.transpose(-1, -2) @ gs).to(v.dtype)
            dp = gs @ vs.transpose(-1, -2)
            ds = 2.0 * s * inv * (dp - (gs * y).sum(-1, keepdim=True))
            dq[b, h] = (ds @ ks).to(q.dtype)
            dk[b, h] = (ds.transpose(-1, -2) @ qs).to(k.dtype)
    out = out.reshape(B, H, Tq, d)
    if grad:
        return out, dq.reshape(B, H, Tq, d), dk, dv
    return out


def _run_plain(st):
    case = st["case"]
    if case["op"] in ("cross", "cross_grad"):
        return _plain_cross(st, case["op"] == "cross_grad")
    cos, sin = _angles(st)
    it = case["inter"]
    yq = _plain_norm(st["q"], st["wq"], cos, sin, it)
    yk = _plain_norm(st["k"], st["wk"], cos, sin, it)
    if case["op"] == "norm":
        return yq, yk
    dq, dwq = _plain_norm_grad(st["gq"], st["q"], st["wq"], cos, sin, it)
    dk, dwk = _plain_norm_grad(st["gk"], st["k"], st["wk"], cos, sin, it)
    return yq, yk, dq, dk, dwq, dwk


# ------------------------------------------------------- the package's entries

def _run_own(st):
    import kernelized_linear_attention_fwd_b200 as K

    case = st["case"]
    if case["op"] in ("norm", "norm_grad"):
        kw = dict(q_weight=st["wq"], k_weight=st["wk"], inv_freq=st["inv_freq"],
                  positions=st["pos"], eps=_EPS, interleaved=case["inter"])
        yq, yk = K.kata_qk_norm_rotate(st["q"], st["k"], **kw)
        if case["op"] == "norm":
            return yq, yk
        return (yq, yk) + tuple(
            K.kata_qk_norm_rotate_backward(st["gq"], st["gk"], st["q"], st["k"], **kw))
    q, k, v, n = st["q"], st["k"], st["v"], st["len"]
    if case["op"] == "cross":
        return K.kata_cross_forward(q, k, v, key_lengths=n)
    y = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    den = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    out = K.kata_cross_forward(q, k, v, key_lengths=n, y_out=y, den_out=den)
    return (out,) + tuple(K.kata_cross_backward(st["g"], q, k, v, y, den, key_lengths=n))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------- work

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    B, H, Hk, d = case["B"], case["H"], case["Hk"], case["d"]
    if case["op"] in ("norm", "norm_grad"):
        T = case["T"]
        n = B * T * (H + Hk) * d
        nbytes = 2 * n * es + 8 * B * T + 8 * d + 2 * case["rot"]
        flops = 8 * n
        if case["op"] == "norm_grad":
            # reads the gradient too (the input once for both), writes dx, dw
            nbytes += 2 * n * es + 8 * d
            flops += 16 * n
        return {"bytes": nbytes, "flops": flops}
    Tq, Tk = case["Tq"], case["Tk"]
    keys = sum(_lengths(case))
    pairs = H * Tq * keys
    rows = B * H * Tq * d
    kv = 2 * Hk * keys * d
    nbytes = 2 * rows * es + kv * es + 4 * B
    flops = 4 * d * pairs
    if case["op"] == "cross_grad":
        # also reads the output's gradient; writes dq and all of dk, dv
        nbytes += 2 * rows * es + 2 * B * Hk * Tk * d * es
        flops += 8 * d * pairs
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------- exact

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("norm", "norm_grad"):
        return _exact_norm(case, st)
    return _exact_cross(case, st)


def _exact_norm(case, st):
    """The rotation as a complex product, sequence by sequence, in 64 bits."""
    n, it = case["rot"] // 2, case["inter"]
    outs = []
    for x, w, gname in ((st["q"], st["wq"], "gq"), (st["k"], st["wk"], "gk")):
        B, T, H, d = x.shape
        w = w.double()
        idx = torch.arange(2 * n, device=x.device)
        first, second = (idx[0::2], idx[1::2]) if it else (idx[:n], idx[n:])
        y = torch.empty(B, H, T, d, dtype=torch.float64, device=x.device)
        dx = torch.empty(B, T, H, d, dtype=torch.float64, device=x.device)
        dw = torch.zeros(d, dtype=torch.float64, device=x.device)
        for b in range(B):
            e = torch.polar(torch.ones(T, n, dtype=torch.float64, device=x.device),
                            torch.outer(st["pos"][b].double(), st["inv_freq"].double()))[:, None]
            X = x[b].double()
            ms = (X ** 2).sum(-1, keepdim=True) / d + _EPS
            hat = X / ms.sqrt()
            z = hat * w
            zr = torch.complex(z[..., first], z[..., second]) * e
            z[..., first], z[..., second] = zr.real, zr.imag
            y[b] = z.transpose(0, 1)
            if case["op"] == "norm_grad":
                G = st[gname][b].double().transpose(0, 1).contiguous()
                gr = torch.complex(G[..., first], G[..., second]) * e.conj()
                G[..., first], G[..., second] = gr.real, gr.imag
                dw += (G * hat).sum((0, 1))
                gz = G * w
                dx[b] = gz / ms.sqrt() - X * (gz * X).sum(-1, keepdim=True) / (d * ms ** 1.5)
        outs.append((y, dx, dw))
    (yq, dq, dwq), (yk, dk, dwk) = outs
    if case["op"] == "norm":
        return yq, yk
    return yq, yk, dq, dk, dwq, dwk


def _exact_cross(case, st):
    """Head by head over the visible keys only, in 64 bits."""
    B, H, Hk, Tq, Tk, d = (case[x] for x in ("B", "H", "Hk", "Tq", "Tk", "d"))
    grad = case["op"] == "cross_grad"
    dev = st["q"].device
    y = torch.zeros(B, H, Tq, d, dtype=torch.float64, device=dev)
    if grad:
        dq = torch.zeros_like(y)
        dk = torch.zeros(B, Hk, Tk, d, dtype=torch.float64, device=dev)
        dv = torch.zeros_like(dk)
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        for h in range(H):
            hk = h // (H // Hk)
            Kh, Vh = st["k"][b, hk, :n].double(), st["v"][b, hk, :n].double()
            for t0 in range(0, Tq, 4096):
                t = slice(t0, min(Tq, t0 + 4096))
                Q = st["q"][b, h, t].double()
                S = torch.einsum("td,sd->ts", Q, Kh)
                den = (S ** 2).sum(1)
                live = den > 0
                scale = torch.zeros_like(den)
                scale[live] = den[live].reciprocal()
                P = S ** 2 * scale[:, None]
                Y = torch.einsum("ts,sd->td", P, Vh)
                y[b, h, t] = Y
                if grad:
                    G = st["g"][b, h, t].double()
                    dv[b, hk, :n] += torch.einsum("ts,td->sd", P, G)
                    # d y_t / d s_ts = 2 s_ts (v_s - y_t) / den_t
                    E = torch.einsum("td,sd->ts", G, Vh) - torch.einsum("td,td->t", G, Y)[:, None]
                    E = 2 * S * E * scale[:, None]
                    dq[b, h, t] = torch.einsum("ts,sd->td", E, Kh)
                    dk[b, hk, :n] += torch.einsum("ts,td->sd", E, Q)
    return (y, dq, dk, dv) if grad else y
