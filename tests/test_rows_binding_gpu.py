"""What the binding of the operators on rows refuses of GPU tensors, and calls from several host
threads whose launches ask for different amounts of LDS."""
import dataclasses

import pytest
import torch

import activation_sparse_expert_amd as moe
from gpu_helpers import DEV
from test_host_threads_gpu import together
from test_linear_q8_gpu import gen, layer, normal, random_codes

pytestmark = pytest.mark.gpu
F16, F32, I8 = torch.float16, torch.float32, torch.int8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def test_linear_q8_refuses():
    g = gen(81)
    lin = layer(g, 24, 64, True, True, "silu")
    q, s = random_codes(g, (5, 64)), torch.ones(5, device=DEV)
    x, y = normal(g, (5, 64), F16), torch.empty((5, 24), dtype=F16, device=DEV)
    for bad in (dict(), dict(x_scale=s[:4]), dict(x_scale=s.half()), dict(x_scale=s.cpu()), dict(x_scale=s, y=y[:4]),
                dict(x_scale=s, y=y, residual=y.float()), dict(x_scale=s, residual=y), dict(x_scale=s, y=y.cpu()),
                dict(x_scale=s, ws=torch.empty(64)), dict(x_scale=s, out_dtype=torch.float64),
                dict(x_scale=torch.ones(10, device=DEV)[::2])):
        with pytest.raises((ValueError, TypeError)):
            moe.linear_q8_forward(lin, q, **bad)
    for change in (dict(bias=lin.bias.half()), dict(w_gate=lin.w_gate[:, :48]), dict(w_gate=None), dict(gate_scale=None),
                   dict(bias_gate=lin.bias_gate[1:]), dict(w=lin.w.t().contiguous().t()), dict(w=lin.w.half()),
                   dict(w_scale=lin.w_scale[1:]), dict(w_scale=lin.w_scale.double()), dict(act="swish")):
        with pytest.raises((ValueError, TypeError)):
            moe.linear_q8_forward(dataclasses.replace(lin, **change), q, x_scale=s)
    for bad, kw in ((x, dict(x_scale=s)), (x.double(), {}), (x[:, :48], {}), (x.t().contiguous().t(), {})):
        with pytest.raises((ValueError, TypeError)):
            moe.linear_q8_forward(lin, bad, **kw)
    for bad, kw in ((x[:0], {}), (x[:1].expand(5, 64), {}), (normal(g, (5, 72), F16)[:, :64], {}),
                    (normal(g, (5, 65), F16).flatten()[1:321].view(5, 64), {}), (q.flatten()[8:].new_zeros(5, 72)[:, :64], dict(x_scale=s))):
        with pytest.raises(moe.MoeError):
            moe.linear_q8_forward(lin, bad, **kw)
    torch.cuda.synchronize()


def test_rows_refuse():
    g = gen(82)
    x, q, s = normal(g, (5, 40), F16), random_codes(g, (5, 40)), torch.ones(5, device=DEV)
    for bad in (dict(q=q[:4]), dict(q=q.half()), dict(q=q.cpu()), dict(scale=s[:4]), dict(scale=s.half()),
                dict(scale=torch.ones(10, device=DEV)[::2]), dict(q=q.t().contiguous().t())):
        with pytest.raises((ValueError, TypeError)):
            moe.quantize_rows(x, **bad)
    for bad in (x.double(), q, x.t().contiguous().t()):
        with pytest.raises((ValueError, TypeError, moe.MoeError)):
            moe.quantize_rows(bad)
    with pytest.raises(moe.MoeError):
        moe.quantize_rows(x[:0])
    for bad in (dict(y=x[:4]), dict(y=x.cpu()), dict(y=x.t().contiguous().t()), dict(out_dtype=torch.float64)):
        with pytest.raises((ValueError, TypeError)):
            moe.dequantize_rows(q, s, **bad)
    for bad in ((q.half(), s), (q, s[:4]), (q, s.half()), (q.t().contiguous().t(), s)):
        with pytest.raises((ValueError, TypeError)):
            moe.dequantize_rows(*bad)
    with pytest.raises(moe.MoeError):
        moe.dequantize_rows(q, s, y=q)
    torch.cuda.synchronize()


def test_norm_refuses():
    g = gen(83)
    r, o = normal(g, (5, 40), F16), normal(g, (5, 40), torch.bfloat16)
    w = torch.ones(40, device=DEV)
    norm = moe.Norm(40, w=w)
    for bad in (dict(y=r[:4]), dict(y=r.float()), dict(y=r.cpu()), dict(out=r[:4]), dict(out=r.cpu()), dict(out=r.t().contiguous().t()),
                dict(gate=r), dict(gate=o[:4]), dict(gate=o[0][:39]), dict(out_dtype=torch.float64),
                dict(out_dtype=I8, out_scale=w[:4]), dict(out_dtype=I8, out_scale=w[:5].half())):
        with pytest.raises((ValueError, TypeError)):
            moe.norm_forward(norm, r, o, **bad)
    for bad in (moe.Norm(39), moe.Norm(40, w=w[:39]), moe.Norm(40, w=w.cpu()), moe.Norm(40, w=w, b=w.half()),
                moe.Norm(40, w=w.double()), moe.Norm(40, w=torch.ones(80, device=DEV)[::2]), moe.Norm(40, kind="group")):
        with pytest.raises((ValueError, TypeError)):
            moe.norm_forward(bad, r, o)
    with pytest.raises(ValueError):
        moe.norm_forward(norm, r, o[:4])
    with pytest.raises(ValueError):
        moe.norm_forward(norm, r, gate=o)
    for kw in (dict(y=o), dict(out=r), dict(out=o), dict(y=r, out=r), dict(out_scale=w[:5]), dict(out=False, y=False)):
        if kw.get("y") is o:                            # y has the residual's type
            kw = dict(y=o.view(F16))
        with pytest.raises(moe.MoeError):
            moe.norm_forward(norm, r, o, **kw)
    for bad in (moe.Norm(40, eps=0.0), moe.Norm(40, post_w=w)):
        with pytest.raises(moe.MoeError):
            moe.norm_forward(bad, r, o)
    with pytest.raises(moe.MoeError):
        moe.norm_forward(moe.Norm(40, post=True), r)
    with pytest.raises(moe.MoeError):
        moe.norm_forward(norm, r[:0])
    torch.cuda.synchronize()


def test_calls_from_several_threads():
    """Streams of 2, 4 and 8 slices, tokens of other lengths made codes of in LDS, tiles, norms."""
    g = gen(84)
    calls = []
    for T, k, n in ((32, 2048, 704), (32, 4096, 9000), (1, 4096, 512), (1, 12288, 704), (1, 4096, 14336), (70, 4096, 2048)):
        lin = layer(g, n, k, bias=True, act="silu")
        x = normal(g, (T, k), torch.bfloat16)
        calls.append(lambda lin=lin, x=x: moe.linear_q8_forward(lin, x))
    norm = moe.Norm(4096, w=normal(g, (4096,), torch.bfloat16), post=True)
    r, o = normal(g, (40, 4096), torch.bfloat16), normal(g, (40, 4096), torch.bfloat16)
    calls.append(lambda: moe.norm_forward(norm, r, o, out_dtype=torch.float32)[1])
    alone = [c() for c in calls]
    torch.cuda.synchronize()
    got = together(calls, 200)
    assert all(torch.equal(a, b) for a, b in zip(alone, got))
