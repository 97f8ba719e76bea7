"""64-bit forms of the linear layer and the dense MoE layer for the GPU tests,
each with a bound of what fp32 sums and the stated roundings may be off.

Bounds.  u = 2^-23 covers one fp32 rounding or truncation.  A product of K terms
is summed in runs of 16 or 32 inside the matrix instruction, at most K / 16
times one after another, and at most 32 partial sums are added at the end: each of
these rounds a value of at most S = sum |x||w| once, so the product is off by
at most (K / 16 + 64) u S.  An activation has a slope of at most 1.13 and is
itself evaluated to a few units of its argument (2^-20 |v| is taken).  The
result is rounded once: eps / 2 relative, or half the smallest subnormal."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -23
SLOPE = 1.13
EVAL = 2.0 ** -20


def act64(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2.0))
    if act == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "silu":
        return v * torch.sigmoid(v)
    return v


def product(x, w, b=None):
    """(x w^T + b, its bound), both fp64."""
    a = x.double() @ w.double().t().contiguous()
    s = x.double().abs() @ w.double().abs().t().contiguous()
    if b is not None:
        a, s = a + b.double(), s + b.double().abs()
    return a, (x.shape[1] / 16 + 64) * U * s


def half_step(y, dtype):
    """Half a rounding step of y in dtype."""
    fi = torch.finfo(dtype)
    return y.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def linear64(x, w, b=None, wg=None, bg=None, act="none", residual=None, out=torch.float32):
    """(y, bound) of the linear layer."""
    a, ea = product(x, w, b)
    if wg is not None:
        g, eg = product(x, wg, bg)
        v = act64(g, act)
        ev = SLOPE * eg + EVAL * g.abs()
        y, e = a * v, ea * v.abs() + ev * (a.abs() + ea)
    else:
        y = act64(a, act)
        e = SLOPE * ea + EVAL * a.abs() if act != "none" else ea
    e = e + U * y.abs()
    if residual is not None:
        y = y + residual.double()
        e = e + U * y.abs()
    return y, e + half_step(y.abs() + e, out)


def choose64(x, router, bias, k, renorm):
    """fp64 logits, the k choices (ties to the lower index) and their weights."""
    lg = x.double() @ router.double().t().contiguous()
    if bias is not None:
        lg = lg + bias.double()
    top, idx = torch.sort(lg, dim=1, descending=True, stable=True)
    e = torch.exp(lg - top[:, :1])
    c = torch.gather(e, 1, idx[:, :k])
    return lg, idx[:, :k], c / (c if renorm else e).sum(1, keepdim=True)


def few64(x, gate, up, down_t, idx, w, n_shared, residual=None, out=torch.float32):
    """(y, bound) of the dense MoE layer with choices idx [T][k] and weights w;
    the shared experts are the last n_shared."""
    T, d = x.shape
    E = gate.shape[0] - n_shared
    y = torch.zeros((T, d), dtype=torch.float64, device=x.device)
    err = torch.zeros_like(y)
    size = torch.zeros_like(y)
    hb = 2.0 ** -17 if x.dtype == torch.bfloat16 else 2.0 ** -21
    idx = idx.cpu().tolist()
    pairs = [(t, e, s) for t in range(T) for s, e in enumerate(idx[t])]
    pairs += [(t, e, None) for t in range(T) for e in range(E, E + n_shared)]
    for e in sorted({p[1] for p in pairs}):
        mine = [p for p in pairs if p[1] == e]
        at = torch.tensor([p[0] for p in mine], device=x.device)
        sc = torch.stack([w[p[0], p[2]].double() if p[2] is not None else
                          torch.ones((), dtype=torch.float64, device=x.device) for p in mine])[:, None]
        g, eg = product(x[at], gate[e])
        a, ea = product(x[at], up[e])
        v = act64(g, "silu")
        h = v * a
        eh = ea * v.abs() + (SLOPE * eg + EVAL * g.abs()) * (a.abs() + ea) + U * h.abs()
        eh = eh + hb * (h.abs() + eh) + 2.0 ** -25       # two 16-bit parts; fp16's subnormals
        wd = down_t[e].double().t().contiguous()
        o, so = h @ wd, (h.abs() + eh) @ wd.abs()
        eo = eh @ wd.abs() + (gate.shape[1] / 16 + 64) * U * so
        y.index_add_(0, at, sc * o)
        err.index_add_(0, at, sc * (eo + 8 * U * so))    # the weight: fp32, a few units
        size.index_add_(0, at, sc * so)
    n_add = len(idx[0]) + n_shared + 16
    err = err + n_add * U * size                         # experts and waves added one by one
    if residual is not None:
        y = y + residual.double()
        err = err + U * y.abs()
    return y, err + half_step(y.abs() + err, out)


def check(got, want, bound, what=""):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst {float((off / bound).max()):.3g} bounds")
