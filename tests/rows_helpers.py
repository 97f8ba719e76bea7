"""64-bit forms of 8-bit rows, the linear layer on them and the norms between two blocks, each
with a bound of what fp32 arithmetic and the stated roundings may be off.

u = 2^-24 is one fp32 rounding relative to its value; U = 2 u.  A sum of d values by one
workgroup goes through at most d / 64 + 16 additions one after another (64 lanes at least
take part), so it is off by at most that many u of the sum of the magnitudes."""
from __future__ import annotations

import torch

from dense_helpers import EVAL, SLOPE, U, act64, half_step

u = U / 2


def codes64(x):
    """Codes and scales of exact arithmetic: 127 x has at most 31 bits and a quotient in fp64 that
    is no tie is at least 2^-32 of itself away from one."""
    v = x.double()
    top = v.abs().amax(1, keepdim=True)
    q = torch.round(127 * v / torch.where(top > 0, top, torch.ones_like(top)))
    return q.to(torch.int8), (top / 127).float()[:, 0]


def linear_q8_64(q, sx, lin, residual=None, out=torch.float32):
    """(y, bound): the sums are integers below 2^31 and exact; one rounding to fp32, two products
    with scales, one addition."""
    def product(w, sw, b):
        a = (q.double() @ w.double().t().contiguous()) * sx.double()[:, None] * sw.double()
        s = a.abs()
        if b is not None:
            a, s = a + b.double(), s + b.double().abs()
        return a, 4 * u * s

    a, ea = product(lin.w, lin.w_scale, lin.bias)
    if lin.w_gate is not None:
        g, eg = product(lin.w_gate, lin.gate_scale, lin.bias_gate)
        v = act64(g, lin.act)
        ev = SLOPE * eg + EVAL * g.abs()
        y, e = a * v, ea * v.abs() + ev * (a.abs() + ea)
    else:
        y = act64(a, lin.act)
        e = SLOPE * ea + EVAL * a.abs() if lin.act != "none" else ea
    e = e + U * y.abs()
    if residual is not None:
        y = y + residual.double()
        e = e + U * y.abs()
    return y, e + half_step(y.abs() + e, out)


def _norm64(z, ez, norm, w, b):
    """(N(z), bound) of rows z that are off by ez."""
    d = z.shape[1]
    chain = d / 64 + 16
    c, ec = z, ez
    if norm.kind == "layer":
        c = z - z.mean(1, keepdim=True)
        ec = ez + ez.mean(1, keepdim=True) + (chain + 2) * u * z.abs().mean(1, keepdim=True) + u * c.abs()
    f = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + norm.eps)
    n = c * f
    # 1 / sqrt halves the relative error of the sum of squares (chain + 2 roundings and what c
    # is off by), and is rounded a few times itself
    en = ec * f + n.abs() * ((chain / 2 + 8) * u + f * f * (c.abs() * ec).mean(1, keepdim=True))
    if w is not None:
        k = w.double() + (1 if norm.offset else 0)
        n, en = n * k, en * k.abs() + 2 * u * (n * k).abs() + u * n.abs() * k.abs()
    if b is not None:
        n = n + b.double()
        en = en + 2 * u * (n.abs() + b.double().abs())
    return n, en


def norm64(norm, residual, block=None, gate=None):
    """(v, its bound, N(v), its bound) before the roundings to the outputs' types."""
    x = residual if residual is not None else block
    v = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    e = torch.zeros_like(v)
    if residual is not None:
        v = norm.residual_scale * residual.double()
        e = 2 * u * v.abs()
    if block is not None:
        c, ec = block.double(), torch.zeros_like(v)
        if norm.post:
            c, ec = _norm64(c, ec, norm, norm.post_w, norm.post_b)
        k = norm.block_scale * (gate.double() if gate is not None else 1)
        if not torch.is_tensor(k):
            k = torch.tensor(k, dtype=torch.float64, device=x.device)
        e = e + ec * k.abs() + 4 * u * (c * k).abs()
        v = v + c * k
        e = e + u * v.abs()
    n, en = _norm64(v, e, norm, norm.w, norm.b)
    return v, e, n, en
