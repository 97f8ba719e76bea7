"""What the binding refuses of GPU tensors before the library is called."""
import dataclasses

import pytest
import torch

import activation_sparse_expert_amd as moe
from gpu_helpers import DEV
from test_few_gpu import make
from test_linear_gpu import gen, layer, normal

pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def few():
    g = gen(71)
    return make(g, 64, 40, 6, 2, 1, F16, bias=True), normal(g, (3, 64), 1.0, F16)


@pytest.mark.parametrize("name", ["router_w", "gate_t", "up_dense", "down_dense"])
def test_few_needs_its_weights(name):
    L, x = few()
    with pytest.raises(ValueError, match="needs router_w, gate_t, up_dense and down_dense"):
        moe.layer_forward_few(dataclasses.replace(L, **{name: None}), x)


@pytest.mark.parametrize("name,change,error", [
    ("router_w", lambda t: t[:, :56], ValueError), ("router_w", lambda t: t.cpu(), ValueError),
    ("router_bias", lambda t: t.half(), TypeError), ("gate_t", lambda t: t[:-1], ValueError),
    ("up_dense", lambda t: t.bfloat16(), TypeError), ("down_dense", lambda t: t.transpose(1, 2), ValueError),
    ("up_dense", lambda t: t.repeat(1, 1, 2)[:, :, ::2], ValueError)])
def test_few_refuses_other_weights(name, change, error):
    L, x = few()
    with pytest.raises(error):
        moe.layer_forward_few(dataclasses.replace(L, **{name: change(getattr(L, name))}), x)


def test_few_refuses_other_inputs_outputs_and_exports():
    L, x = few()
    y = torch.empty((3, 64), dtype=F16, device=DEV)
    for bad in (dict(y=y[:2]), dict(y=y, residual=x.float()), dict(residual=x), dict(y=y, residual=x[:, :32]),
                dict(y=y.cpu()), dict(trace={"masks": y}), dict(trace={"topk_idx": torch.empty((3, 2), device=DEV)}),
                dict(trace={"logits": torch.empty((3, 5), device=DEV)}), dict(ws=torch.empty(64)),
                dict(out_dtype=torch.float64)):
        with pytest.raises((ValueError, TypeError)):
            moe.layer_forward_few(L, x, **bad)
    with pytest.raises(ValueError):
        moe.layer_forward_few(L, x[:, :32])
    with pytest.raises(ValueError):
        moe.layer_forward_few(L, x.t().contiguous().t())
    for bad in (x[:0], x.bfloat16(), x.repeat(11, 1)):
        with pytest.raises(moe.MoeError):
            moe.layer_forward_few(L, bad)


def test_linear_refuses():
    g = gen(72)
    lin = layer(g, 24, 64, F16, True, True, "silu")
    x = normal(g, (5, 64), 1.0, F16)
    y = torch.empty((5, 24), dtype=F16, device=DEV)
    for bad in (dict(y=y[:4]), dict(y=y, residual=y.float()), dict(residual=y), dict(y=y.cpu()), dict(ws=torch.empty(64)),
                dict(y=y.t().contiguous().t()), dict(out_dtype=torch.float64)):
        with pytest.raises((ValueError, TypeError)):
            moe.linear_forward(lin, x, **bad)
    for change in (dict(bias=lin.bias.half()), dict(w_gate=lin.w_gate[:, :56]), dict(bias_gate=lin.bias_gate[1:]),
                   dict(w=lin.w.t().contiguous().t()), dict(w_gate=lin.w_gate.bfloat16()), dict(act="swish")):
        with pytest.raises((ValueError, TypeError)):
            moe.linear_forward(dataclasses.replace(lin, **change), x)
    for bad in (x[:0], x.bfloat16(), x[:1].expand(5, 64), normal(g, (5, 68), 1.0, F16)[:, :64],
                normal(g, (5, 65), 1.0, F16).flatten()[1:321].view(5, 64)):
        with pytest.raises(moe.MoeError):
            moe.linear_forward(lin, bad)
    square = layer(g, 64, 64, F16)
    with pytest.raises(moe.MoeError):
        moe.linear_forward(square, x, y=x)
    torch.cuda.synchronize()
