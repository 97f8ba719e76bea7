"""Refusals of the linear layer and the few-token MoE layer, without a GPU."""
import ctypes as C

import pytest
import torch

import activation_sparse_expert_amd as moe
from test_api_host import FAKE, _lib_or_skip


def _linear(n=704, k=256, wdt=0, w=FAKE, bias=None, w_gate=None, bias_gate=None, act=0, x=FAKE, xdt=0, xs=None,
            T=4, r=None, rs=None, y=FAKE, ydt=2, ys=None, ws=FAKE, ws_bytes=1 << 28):
    L = _lib_or_skip()
    dsc = moe.LinearDesc(n, k, wdt, w, bias, w_gate, bias_gate, act)
    return L.moe_linear_forward(C.byref(dsc), x, xdt, k if xs is None else xs, T, r, n if rs is None else rs, y,
                                ydt, n if ys is None else ys, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(y=None), -1), (dict(w=None), -1), (dict(T=0), -1), (dict(T=65537), -1),
    (dict(n=0), -1), (dict(k=0), -1), (dict(act=5), -1), (dict(act=-1), -1), (dict(bias_gate=FAKE), -1),
    (dict(xs=248), -1), (dict(ys=703), -1), (dict(r=FAKE + 65536, rs=700), -1),
    (dict(r=FAKE, rs=800), -1),                 # residual is y, at another stride
    (dict(k=260), -2), (dict(k=4, xs=8), -2), (dict(wdt=2), -2), (dict(xdt=1), -2), (dict(ydt=3), -2),
    (dict(k=(1 << 20) + 8), -2), (dict(n=(1 << 24) + 1), -2),
    (dict(x=FAKE + 8), -3), (dict(xs=260), -3), (dict(w=FAKE + 2), -3), (dict(w_gate=FAKE + 8), -3),
    (dict(y=FAKE + 2), -3), (dict(r=FAKE + 2), -3), (dict(bias=FAKE + 2), -3),
    (dict(w_gate=FAKE, bias_gate=FAKE + 1), -3),
    (dict(T=40, k=16384, n=64, ws=None), -4), (dict(T=40, k=16384, n=64, ws_bytes=0), -4),
    (dict(T=40, k=16384, n=64, ws_bytes=256), -4), (dict(ws=FAKE + 4), -3),
])
def test_linear_rejects(kw, code):
    assert _linear(**kw) == code


def test_linear_null_layer():
    L = _lib_or_skip()
    assert L.moe_linear_forward(None, FAKE, 0, 256, 1, None, 0, FAKE, 2, 704, FAKE, 1 << 20, None) == -1


def _desc(**kw):
    base = dict(d=2048, f=1408, n_routed=64, n_shared=2, top_k=6, renormalize=1, wdt=0, router_w=FAKE, rdt=0,
                router_bias=None, up_q=None, up_sz=None, gate_t=FAKE, down=None, thresholds=None, up_dense=FAKE,
                down_dense=FAKE, density=0.0)
    base.update(kw)
    return moe.LayerDesc(*[base[n] for n, _ in moe.LayerDesc._fields_])


def _few(x=FAKE, xdt=0, T=4, r=None, y=FAKE, ydt=2, trace=None, ws=FAKE, ws_bytes=1 << 28, **kw):
    L = _lib_or_skip()
    dsc = _desc(**kw)
    return L.moe_layer_forward_few(C.byref(dsc), x, xdt, T, r, y, ydt, C.byref(trace) if trace else None, ws,
                                   ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(y=None), -1), (dict(T=0), -1), (dict(T=33), -2), (dict(n_shared=-1), -1),
    (dict(top_k=0), -1), (dict(top_k=65), -1), (dict(f=0), -1), (dict(f=1404), -2), (dict(d=2044), -2),
    (dict(d=16392), -2), (dict(T=32, top_k=64), -2), (dict(n_routed=2000), -1), (dict(n_shared=2000, T=2), -2),
    (dict(router_w=None), -1), (dict(gate_t=None), -1), (dict(up_dense=None), -1), (dict(down_dense=None), -1),
    (dict(wdt=2), -2), (dict(xdt=1), -2), (dict(ydt=4), -2), (dict(rdt=3), -2),
    (dict(x=FAKE + 8), -3), (dict(gate_t=FAKE + 8), -3), (dict(up_dense=FAKE + 2), -3),
    (dict(down_dense=FAKE + 4), -3), (dict(router_w=FAKE + 2), -3), (dict(router_bias=FAKE + 2), -3),
    (dict(y=FAKE + 2), -3), (dict(r=FAKE + 2), -3),
    (dict(ws=None), -4), (dict(ws_bytes=4096), -4), (dict(ws=FAKE + 8), -3),
])
def test_few_rejects(kw, code):
    assert _few(**kw) == code


@pytest.mark.parametrize("field,val,code", [
    ("masks", FAKE, -2), ("mask_bits", FAKE, -2), ("nnz", FAKE, -2), ("topk_idx", FAKE + 2, -3),
    ("topk_w", FAKE + 1, -3), ("logits", FAKE + 2, -3), ("expert_count", FAKE + 2, -3), ("eam_row", FAKE + 2, -3),
])
def test_few_trace_rejects(field, val, code):
    assert _few(trace=moe.LayerTrace(**{field: val})) == code


def test_workspace_sizes():
    _lib_or_skip()
    assert moe.workspace_size(moe.OP_LINEAR, 1, 256, 704) == 0          # needs none
    assert moe.workspace_size(moe.OP_LINEAR, 1, 260, 704) == 0
    assert moe.workspace_size(moe.OP_LINEAR, 65537, 256, 704) == 0
    # a split of K keeps at least two fp32 products
    assert moe.workspace_size(moe.OP_LINEAR, 64, 16384, 64) >= 2 * 64 * 64 * 4
    few = moe.workspace_size(moe.OP_LAYER_FEW, 32, 2048, 1408, 64, 6, 2)
    assert few >= 32 * 8 * 1408 * 4
    assert moe.workspace_size(moe.OP_LAYER_FEW, 33, 2048, 1408, 64, 6, 2) == 0
    assert moe.workspace_size(moe.OP_LAYER_FEW, 1, 2048, 1408, 64, 65, 2) == 0


def test_binding_checks_before_the_library():
    """Shapes, types and devices are refused in Python (CPU tensors here)."""
    w = torch.zeros((16, 8), dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.linear_forward(moe.Linear(w), torch.zeros((2, 8), dtype=torch.float16))
    with pytest.raises(ValueError, match=r"\[T\]\[k\]"):
        moe.linear_forward(moe.Linear(w), torch.zeros(8, dtype=torch.float16))
    with pytest.raises(ValueError, match="act"):
        moe.Linear(w, act="tanh").desc()
    with pytest.raises(ValueError, match=r"\[T\]\[d\]"):
        moe.layer_forward_few(None, torch.zeros(8, dtype=torch.float16))


@pytest.mark.parametrize("kw,code", [
    (dict(T=32, d=16384, top_k=2, ws_bytes=0), -4), (dict(T=32, d=16392, top_k=2), -2), (dict(T=33), -2),
    (dict(T=32, top_k=62, ws_bytes=0), -4), (dict(T=32, top_k=63), -2),
    (dict(n_routed=1024, ws_bytes=0), -4), (dict(n_routed=1025), -1), (dict(n_routed=4, top_k=5), -1),
])
def test_few_limits_are_the_documented_ones(kw, code):
    """Both sides of each limit; on the near side the workspace is what is missing."""
    assert _few(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=65536, ws=FAKE + 8), -3), (dict(T=65537), -1), (dict(k=1 << 20, T=40, ws_bytes=0), -4),
    (dict(k=(1 << 20) + 8), -2), (dict(n=(1 << 24) + 1), -2),
])
def test_linear_limits_are_the_documented_ones(kw, code):
    """Both sides of each limit; on the near side it is the workspace that is refused."""
    assert _linear(**kw) == code


def test_linear_refuses_its_input_as_output():
    assert _linear(T=1, n=256, k=256, ws=None, ws_bytes=0) == -1
    assert _linear(T=40, n=256, k=256) == -1
