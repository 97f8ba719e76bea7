"""Refusals of the operators on rows of tokens, without a GPU."""
import ctypes as C

import pytest
import torch

import activation_sparse_expert_amd as moe
from test_api_host import FAKE, _lib_or_skip

F2, F3 = FAKE + (1 << 20), FAKE + (2 << 20)


def _linear(n=704, k=256, w=FAKE, sw=FAKE, bias=None, wg=None, sg=None, bias_gate=None, act=0, x=F2, xdt=3, xs=None, sx=FAKE,
            T=4, r=None, rs=None, y=FAKE, ydt=2, ys=None, ws=FAKE, ws_bytes=1 << 28):
    L = _lib_or_skip()
    dsc = moe.LinearQ8Desc(n, k, w, sw, bias, wg, sg, bias_gate, act)
    return L.moe_linear_q8_forward(C.byref(dsc), x, xdt, k if xs is None else xs, sx, T, r, n if rs is None else rs, y,
                                   ydt, n if ys is None else ys, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(y=None), -1), (dict(w=None), -1), (dict(sw=None), -1), (dict(T=0), -1), (dict(T=65537), -1),
    (dict(n=0), -1), (dict(k=0), -1), (dict(act=5), -1), (dict(act=-1), -1), (dict(bias_gate=FAKE), -1),
    (dict(wg=FAKE), -1), (dict(sg=FAKE), -1),           # gate weights and their scales come together
    (dict(sx=None), -1), (dict(xdt=0), -1), (dict(xdt=2), -1),      # codes have scales, other types none
    (dict(xs=240), -1), (dict(ys=703), -1), (dict(r=F3, rs=700), -1), (dict(r=FAKE, rs=800), -1),
    (dict(x=FAKE), -1),                                 # x is y
    (dict(k=264), -2), (dict(k=8, xs=16), -2), (dict(xdt=4), -2), (dict(ydt=3), -2), (dict(xdt=-1), -2),
    (dict(k=1 << 17), -2), (dict(n=(1 << 24) + 1), -2),
    (dict(x=F2 + 8), -3), (dict(xs=264), -3), (dict(w=FAKE + 8), -3), (dict(wg=FAKE + 8, sg=FAKE), -3),
    (dict(wg=FAKE, sg=FAKE + 2), -3), (dict(sw=FAKE + 2), -3), (dict(sx=FAKE + 1), -3),
    (dict(y=FAKE + 2), -3), (dict(r=FAKE + 2), -3), (dict(bias=FAKE + 2), -3),
    (dict(wg=FAKE, sg=FAKE, bias_gate=FAKE + 1), -3),
    (dict(xdt=0, sx=None, T=300, k=4096, ws=None), -4), (dict(xdt=1, sx=None, T=300, k=4096, ws_bytes=300 * 4096), -4),
    (dict(ws=FAKE + 4), -3),
    # the far side of each limit is above; on the near side it is the workspace or an address that is refused
    (dict(T=65536, ws=FAKE + 8), -3), (dict(k=(1 << 17) - 16, xdt=2, sx=None, T=300, ws_bytes=0), -4),
    (dict(n=1 << 24, ws=FAKE + 8), -3), (dict(k=16, ws=FAKE + 8), -3),
])
def test_linear_q8_rejects(kw, code):
    assert _linear(**kw) == code


def test_linear_q8_null_layer_and_workspace():
    L = _lib_or_skip()
    assert L.moe_linear_q8_forward(None, F2, 3, 256, FAKE, 1, None, 0, FAKE, 2, 704, FAKE, 1 << 20, None) == -1
    size = lambda T, k, n, xdt: moe.workspace_size(moe.OP_LINEAR_Q8, T, k, n, xdt, 0, 0)
    assert size(300, 4096, 4096, 0) >= size(300, 4096, 4096, 3) + 300 * 4096 + 300 * 4
    assert size(4, 264, 64, 0) == 0 and size(0, 256, 64, 0) == 0 and size(300, 256, 64, 4) == 0 and size(65537, 256, 64, 0) == 0
    assert size(1, 256, 704, 3) == 0                    # needs none


def _quantize(x=FAKE, xdt=0, xs=None, T=3, k=100, q=F2, qs=None, scale=F3):
    return _lib_or_skip().moe_quantize_rows(x, xdt, k if xs is None else xs, T, k, q, k if qs is None else qs, scale, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(q=None), -1), (dict(scale=None), -1), (dict(T=0), -1), (dict(k=0), -1), (dict(xs=99), -1),
    (dict(qs=99), -1), (dict(q=FAKE), -1), (dict(scale=FAKE), -1), (dict(scale=F2), -1), (dict(k=(1 << 20) + 1), -2),
    (dict(xdt=3), -2), (dict(xdt=-1), -2), (dict(x=FAKE + 1), -3), (dict(x=FAKE + 2, xdt=2), -3), (dict(scale=F3 + 2), -3),
    (dict(k=1 << 20, scale=F3 + 2), -3),
])
def test_quantize_rejects(kw, code):
    assert _quantize(**kw) == code


def _dequantize(q=FAKE, qs=None, scale=F3, T=3, k=100, y=F2, ydt=0, ys=None):
    return _lib_or_skip().moe_dequantize_rows(q, k if qs is None else qs, scale, T, k, y, ydt, k if ys is None else ys, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(y=None), -1), (dict(scale=None), -1), (dict(T=0), -1), (dict(k=0), -1), (dict(qs=99), -1),
    (dict(ys=99), -1), (dict(y=FAKE), -1), (dict(y=F3), -1), (dict(k=(1 << 20) + 1), -2), (dict(ydt=3), -2), (dict(ydt=9), -2),
    (dict(y=F2 + 1), -3), (dict(y=F2 + 2, ydt=2), -3), (dict(scale=F3 + 1), -3),
])
def test_dequantize_rejects(kw, code):
    assert _dequantize(**kw) == code


def _norm(d=256, kind=0, eps=1e-6, wdt=0, w=None, b=None, post=0, pw=None, pb=None, T=4, r=FAKE, rdt=0, rs=None, o=F2, odt=0,
          os=None, g=None, gs=0, y=F3, ys=None, out=F3 + 65536, ndt=0, ns=None, scale=None, null=False):
    dsc = moe.NormDesc(d, kind, eps, wdt, w, b, post, pw, pb, 0, 1.0, 1.0)
    return _lib_or_skip().moe_norm_forward(None if null else C.byref(dsc), T, r, rdt, d if rs is None else rs, o, odt,
                                           d if os is None else os, g, gs, y, d if ys is None else ys, out, ndt,
                                           d if ns is None else ns, scale, None)


@pytest.mark.parametrize("kw,code", [
    (dict(null=True), -1), (dict(T=0), -1), (dict(d=0), -1), (dict(kind=2), -1), (dict(kind=-1), -1),
    (dict(r=None, o=None), -1), (dict(y=None, out=None), -1),
    (dict(eps=0.0), -1), (dict(eps=1e-39), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(eps=-1.0), -1),
    (dict(pw=FAKE), -1), (dict(pb=FAKE), -1), (dict(o=None, post=1), -1), (dict(o=None, g=FAKE), -1),
    (dict(rs=255), -1), (dict(os=255), -1), (dict(ys=255), -1), (dict(ns=255), -1), (dict(g=FAKE, gs=255), -1),
    (dict(y=F2), -1), (dict(y=FAKE, ys=300), -1), (dict(g=F3, gs=256), -1), (dict(out=F3), -1), (dict(out=FAKE), -1),
    (dict(out=F2), -1), (dict(g=F3 + 65536), -1),
    (dict(ndt=3), -1), (dict(scale=FAKE), -1),          # codes have scales, other types none
    (dict(d=16385), -2), (dict(rdt=3), -2), (dict(odt=3), -2), (dict(ndt=4), -2), (dict(w=FAKE, wdt=3), -2),
    (dict(r=None, rdt=7), -2), (dict(ndt=-1), -2),
    (dict(r=FAKE + 1), -3), (dict(r=FAKE + 2, rdt=2), -3), (dict(o=F2 + 1), -3), (dict(g=FAKE + 1), -3), (dict(y=F3 + 1), -3),
    (dict(out=F3 + 65537), -3), (dict(w=FAKE + 1), -3), (dict(b=FAKE + 2, wdt=2), -3), (dict(post=1, pw=FAKE + 1), -3),
    (dict(post=1, pb=FAKE + 1), -3), (dict(ndt=3, scale=FAKE + 2), -3), (dict(d=16384, r=FAKE + 1), -3),
])
def test_norm_rejects(kw, code):
    assert _norm(**kw) == code


def test_binding_checks_before_the_library():
    """Shapes, types and devices are refused in Python (CPU tensors here)."""
    x = torch.zeros((2, 16), dtype=torch.float16)
    w, s = torch.zeros((4, 16), dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.linear_q8_forward(moe.LinearQ8(w, s), x)
    with pytest.raises(ValueError, match=r"\[T\]\[k\]"):
        moe.linear_q8_forward(moe.LinearQ8(w, s), x[0])
    with pytest.raises(ValueError, match="act"):
        moe.LinearQ8(w, s, act="tanh").desc()
    for call in (lambda: moe.quantize_rows(x), lambda: moe.dequantize_rows(w, s), lambda: moe.norm_forward(moe.Norm(16), x)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    for call in (lambda: moe.quantize_rows(x[0]), lambda: moe.dequantize_rows(w[0], s), lambda: moe.norm_forward(moe.Norm(16), x[0])):
        with pytest.raises(ValueError, match="must be"):
            call()
    with pytest.raises(ValueError, match="residual or a block"):
        moe.norm_forward(moe.Norm(16), None)
    with pytest.raises(ValueError, match="kind"):
        moe.Norm(16, kind="batch").desc()
    with pytest.raises(TypeError, match="one dtype"):
        moe.Norm(16, w=x[0], b=s).desc()
