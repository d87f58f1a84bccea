"""Plain 64-bit forms of the head norm with rotation and of cross attention,
with their gradients and elementwise bounds of the kernels' rounding errors.

Torch tensors of any device; everything is computed in float64 from the exact
values of the inputs.
"""
from __future__ import annotations

import torch

# Largest relative error of one rounding: half a step.
HALF = {torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2, torch.float32: torch.finfo(torch.float32).eps / 2}
U = HALF[torch.float32]


# ------------------------------------------------------------------ norm and rotation

def _turn(x, ang, interleaved):
    """x [..., d] turned by ang [..., n] on its pairs."""
    n = ang.shape[-1]
    i = torch.arange(n, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    y = x.clone()
    c, s = ang.cos(), ang.sin()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def angles(positions, inv_freq, B, T, device):
    """[B, 1, T, n] angles; positions None: 0 .. T-1."""
    if inv_freq is None:
        return torch.zeros(B, 1, T, 0, dtype=torch.float64, device=device)
    p = torch.arange(T, device=device) if positions is None else positions
    p = p.double().expand(B, T)
    return (p[..., None] * inv_freq.double())[:, None]


def norm_rotate(x, w, ang, eps, interleaved):
    """y [B, H, T, d] of x [B, T, H, d]."""
    x = x.double().transpose(1, 2)
    u = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt()
    return _turn(u if w is None else u * w.double(), ang, interleaved)


def norm_rotate_grad(gy, x, w, ang, eps, interleaved):
    """(dx [B, T, H, d], dw [d])."""
    x = x.double().transpose(1, 2)
    r = ((x * x).mean(-1, keepdim=True) + eps).rsqrt()
    u = x * r
    g = _turn(gy.double(), -ang, interleaved)
    dw = (g * u).sum((0, 1, 2))
    g = g if w is None else g * w.double()
    dx = r * (g - u * (g * u).mean(-1, keepdim=True))
    return dx.transpose(1, 2), dw


def norm_rotate_bounds(y, x, w, dtype, eps, interleaved, n):
    """Bound of |kernel - y|: the output's rounding, and in fp32 the norm (a sum
    of d <= 64 squares in chains of 8 and 3 additions, its reciprocal root at 2
    steps, three products: below 16 U), the products and the sum of the turn (3 U)
    and the angle (a 32-bit fraction of a half turn, pi 2^-25 < 2 U, and sine
    and cosine at 2 steps each): together below 32 U of both members of the pair."""
    x = x.double().transpose(1, 2)
    z = x.abs() / ((x * x).mean(-1, keepdim=True) + eps).sqrt()
    z = z if w is None else z * w.double().abs()
    i = torch.arange(n, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    m = z.clone()
    m[..., a] = m[..., b] = z[..., a] + z[..., b]
    return HALF[dtype] * y.abs() + 32 * U * m + 1e-30


def norm_grad_bounds(dx, gy, x, w, dtype, eps, interleaved, n):
    """As above: the turn, the norm, two sums of d terms, below 48 U of the sum of
    the magnitudes that enter; dw adds at most 1024 rows in chains (the tests'
    sizes) on 48 U."""
    x = x.double().transpose(1, 2)
    r = ((x * x).mean(-1, keepdim=True) + eps).rsqrt()
    u = (x * r).abs()
    g = gy.double().abs()
    i = torch.arange(n, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    m = g.clone()
    m[..., a] = m[..., b] = g[..., a] + g[..., b]
    dw = (m * u).sum((0, 1, 2))
    m = m if w is None else m * w.double().abs()
    bdx = r * (m + u * (m * u).mean(-1, keepdim=True))
    return HALF[dtype] * dx.abs() + 48 * U * bdx.transpose(1, 2) + 1e-30, (1024 + 48) * U * dw + 1e-30


# ------------------------------------------------------------------ cross attention

def _parts(q, k, v, lengths):
    """(q [B, Hk, R, d], k, v with the masked keys as zeros, visible [B, 1, 1, Tk])."""
    B, H, Tq, d = q.shape
    Hk, Tk = k.shape[1], k.shape[2]
    q = q.double().reshape(B, Hk, (H // Hk) * Tq, d)
    vis = torch.ones(B, Tk, dtype=torch.bool, device=q.device)
    if lengths is not None:
        vis = torch.arange(Tk, device=q.device)[None] < lengths.to(q.device)[:, None]
    zero = torch.zeros((), dtype=torch.float64, device=q.device)
    k = torch.where(vis[:, None, :, None], k.double(), zero)
    v = torch.where(vis[:, None, :, None], v.double(), zero)
    return q, k, v, vis[:, None, None, :]


def cross(q, k, v, lengths=None):
    """(y [B, H, Tq, d], l [B, H, Tq])."""
    qr, kk, vv, _ = _parts(q, k, v, lengths)
    w = (qr @ kk.transpose(-1, -2)) ** 2
    l = w.sum(-1, keepdim=True)
    y = torch.where(l > 0, (w @ vv) / l, torch.zeros_like(l))
    return y.reshape(q.shape), l.reshape(q.shape[:3])


def cross_grad(dout, q, k, v, lengths=None):
    """(dq, dk, dv)."""
    qr, kk, vv, _ = _parts(q, k, v, lengths)
    g = dout.double().reshape(qr.shape)
    s = qr @ kk.transpose(-1, -2)
    l = (s * s).sum(-1, keepdim=True)
    inv = torch.where(l > 0, 1 / l, torch.zeros_like(l))
    y = ((s * s) @ vv) * inv
    c = 2 * s * inv * (g @ vv.transpose(-1, -2) - (g * y).sum(-1, keepdim=True))
    return (c @ kk).reshape(q.shape), c.transpose(-1, -2) @ qr, (s * s * inv).transpose(-1, -2) @ g


def cross_bounds(q, k, v, dtype, lengths=None, dout=None, split=False):
    """Elementwise bounds of the kernels' errors, to first order and times 1.1.

    e is the relative error of an operand that goes back into the products (bf16:
    half a step, or with `split`, as two numbers, that of a half step; fp32: none
    beyond a), a that of a sum relative to the sum of
    its terms' magnitudes: chains of up to 64 terms, then of up to Tk / 64 (fp32) or
    of Tk / 16 (tensor cores, which may truncate: a whole step each).

      s:  a A with A = sum |q_i k_i|            w: 2 |s| a A, and e w
      y:  sum (dw |v - y|) / l + a sum w |v| / l + the output's rounding
    With a gradient also (D = dout.y, p = dout.v, c = 2 s (p - D) / l):
      D:  sum |dout| dy + a sum |dout y|        1 / l: e + a
      c:  |c| (2 e + 4 a) + 2 / l (a A |p - D| + |s| (a P + dD)), P = sum |dout v|
      dq, dk, dv: sums of those against |k|, |q|, |dout|, plus a times the sum of
      magnitudes, plus the output's rounding.
    """
    qr, kk, vv, _ = _parts(q, k, v, lengths)
    Tk, R = kk.shape[2], qr.shape[2]
    e = HALF[dtype] if dtype == torch.bfloat16 else 0.0
    e = e * e if split else e
    n = max(Tk, R)
    a = U * (64 + 8 + (n / 64 if dtype == torch.float32 else 2 * n / 16))
    half = HALF[dtype]
    s = qr @ kk.transpose(-1, -2)
    A = qr.abs() @ kk.abs().transpose(-1, -2)
    w = s * s
    l = w.sum(-1, keepdim=True)
    inv = torch.where(l > 0, 1 / l, torch.zeros_like(l))
    y = (w @ vv) * inv
    dw = e * w + 2 * s.abs() * a * A
    # sum dw |v - y| <= sum dw |v| + |y| sum dw, tighter: take both members per column block
    by = torch.zeros_like(y)
    for c0 in range(0, y.shape[-1], 4):
        by[..., c0:c0 + 4] = torch.einsum("bhrs,bhrsc->bhrc", dw, (
            vv[:, :, None, :, c0:c0 + 4] - y[..., None, c0:c0 + 4]).abs())
    by = by * inv + a * (w @ vv.abs()) * inv
    out = 1.1 * (by + 4 * U * y.abs()) + 1e-30
    if dout is None:
        return (out + half * y.abs()).reshape(q.shape), out.reshape(q.shape)
    g = dout.double().reshape(qr.shape)
    p = g @ vv.transpose(-1, -2)
    P = g.abs() @ vv.abs().transpose(-1, -2)
    D = (g * y).sum(-1, keepdim=True)
    dD = (g.abs() * by).sum(-1, keepdim=True) + a * (g * y).abs().sum(-1, keepdim=True)
    c = 2 * s * inv * (p - D)
    bc = c.abs() * (2 * e + 4 * a) + 2 * inv * (a * A * (p - D).abs() + s.abs() * (a * P + dD))
    pw = w * inv
    bp = pw * (2 * e + 4 * a) + dw * inv
    dq, dk, dv = c @ kk, c.transpose(-1, -2) @ qr, pw.transpose(-1, -2) @ g
    bq = bc @ kk.abs() + a * (c.abs() @ kk.abs())
    bk = (bc + a * c.abs()).transpose(-1, -2) @ qr.abs()
    bv = (bp + a * pw).transpose(-1, -2) @ g.abs()
    return tuple((1.1 * b + half * x.abs() + 1e-30).reshape(t.shape)
                 for b, x, t in ((bq, dq, q), (bk, dk, k), (bv, dv, v)))


def worst(got, want, bound):
    """Largest |got - want| / bound (inf where got is not finite)."""
    got = got.double()
    if got.numel() == 0:
        return 0.0
    r = (got - want).abs() / bound
    return float(torch.where(torch.isfinite(got), r, torch.full_like(r, float("inf"))).max())
