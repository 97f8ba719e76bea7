"""What the few-token layer keeps of h = SiLU(g) u, read off y.

One expert whose W^down is the identity (or a few of its columns), and tokens
that are one input times a unit vector: then g, u and every sum have one term
and are exact, the router weight is 1, and y is h as the layer holds it.

Bounds, in u = 2^-24 (half a unit of fp32) relative to |h|: exp(-g) is off by
at most (2 |g| + 2) u (its argument is rounded twice, in g log2 e), 1 + exp(-g),
the quotient and the product by u by one rounding each, the sums of h's parts
and of the waves by one each: (2 |g| + 10) u.  A part of h has the 16-bit type's
P = 11 (fp16) or 8 (bf16) bits, so its rounding leaves at most 2^-P of what it
rounds; in fp16 a part is at least half a step of 2^-24 exact, and the second and
third part are kept times 2^11 and 2^22."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
BITS = {"f16": 11, "bf16": 8}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def reading(T, f, dt, scale, seed):
    """(layer, x, h in 64 bits, g): x[t] = scale_t e_t, E = 1, W^down the identity."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    d = f
    assert T <= d
    gate = torch.zeros((1, f, d), device=DEV)
    up = torch.zeros((1, f, d), device=DEV)
    gate[0, :, :T] = torch.randn((f, T), generator=g, device=DEV) * scale
    up[0, :, :T] = torch.randn((f, T), generator=g, device=DEV) * scale
    gate, up = gate.to(dt), up.to(dt)
    x = torch.zeros((T, d), device=DEV)
    x[range(T), range(T)] = 2.0 ** torch.randint(-1, 2, (T,), generator=g, device=DEV)
    x = x.to(dt)
    L = moe.Layer(d=d, f=f, E=1, S=0, k=1, renormalize=True, router_w=torch.zeros((1, d), dtype=dt, device=DEV),
                  up_q=None, up_sz=None, thresholds=None, down=None, gate_t=gate, up_dense=up,
                  down_dense=torch.eye(f, device=DEV).to(dt)[None].contiguous())
    g64 = x.double() @ gate[0].double().t().contiguous()
    u64 = x.double() @ up[0].double().t().contiguous()
    return L, x, g64 * torch.sigmoid(g64) * u64, g64


def off(y, h, bound, what):
    e = (y.double() - h).abs()
    worst, within = float((e / bound).max()), bool((e <= bound).all())
    say(f"{what}: worst {worst:.3g} bounds, relative L2 {float(e.norm() / h.norm()):.3g}")
    assert within, f"{what}: {worst:.3g} bounds"


SCALES = [2.0 ** -11, 2.0 ** -9, 2.0 ** -6, 2.0 ** -3, 1.0, 4.0]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 4, 6, 8, 13, 32])
def test_two_parts_of_h_at_every_scale(T, dt):
    """y in 32 bits shows at least h's two parts: 2^-2P, and in fp16 2^-36 for values
    below fp16's normal ones (h from 2^-24 on)."""
    for i, scale in enumerate(SCALES):
        L, x, h, g = reading(T, 200, DT[dt], scale, 10 * T + i)
        y = moe.layer_forward_few(L, x)
        bound = h.abs() * (2.0 ** (-2 * BITS[dt]) + (2 * g.abs() + 10) * U) + (2.0 ** -36 if dt == "f16" else 2.0 ** -126)
        off(y, h, bound, f"T={T} {dt} scale {scale}")


@pytest.mark.parametrize("dt,out", [("f16", torch.float32), ("bf16", torch.float32), ("bf16", torch.float16),
                                    ("f16", torch.bfloat16)])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 6, 8, 9, 10, 13, 16, 17, 27, 32])
def test_outputs_of_another_type_lose_nothing_of_h(T, dt, out):
    """h has 24 bits, as an fp32 h has (in fp16 2^-47 for the smallest)."""
    for i, scale in enumerate(SCALES):
        L, x, h, g = reading(T, 264, DT[dt], scale, 20 * T + i)
        y = moe.layer_forward_few(L, x, out_dtype=out)
        bound = h.abs() * ((2 * g.abs() + 11) * U) + (2.0 ** -47 if dt == "f16" else 2.0 ** -126)
        if out != torch.float32:
            fi = torch.finfo(out)
            bound = bound + h.abs() * fi.eps / 2 * 1.001 + fi.smallest_normal * fi.eps / 2
        off(y, h, bound, f"T={T} {dt} -> {out} scale {scale}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 4, 8, 13, 32])
def test_y_of_the_own_type_is_rounded_once(T, dt):
    """y is h rounded to the layer's type, up to the 24 bits (fp16: 22) that h has: off by
    half a step of y and no more than those."""
    for i, scale in enumerate([2.0 ** -3, 1.0, 4.0]):
        L, x, h, g = reading(T, 264, DT[dt], scale, 30 * T + i)
        y = moe.layer_forward_few(L, x, out_dtype=DT[dt])
        low = -14 if dt == "f16" else -126               # the exponent of the smallest normal value
        step = torch.ldexp(torch.ones_like(h), torch.frexp(h.abs())[1].clamp(min=low + 1) - BITS[dt])
        kept = h.abs() * 2.0 ** -22 + 2.0 ** -36 if dt == "f16" else 2.0 ** -126
        off(y, h, step / 2 + kept + h.abs() * (2 * g.abs() + 11) * U, f"T={T} {dt} scale {scale}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 3, 8, 13, 30])
@pytest.mark.parametrize("own", [True, False])
def test_infinite_down_weights_give_what_the_formula_gives(T, dt, own):
    """An infinity of W^down times a finite h other than 0 is an infinity of the
    product's sign, whatever the parts that h is kept in; the other outputs are as
    without it, and two infinities of opposite sign make a NaN."""
    f = 136
    L, x, h, g = reading(T, f, DT[dt], 1.0, 3 + T)
    out = DT[dt] if own else torch.float32
    clean = moe.layer_forward_few(L, x, out_dtype=out)
    assert float(h.abs().min()) > 2.0 ** -25            # the first part of none is 0 (fp16's step is 2^-24)
    inf = float("inf")
    L.down_dense[0, 5, 77] = inf
    L.down_dense[0, 130, 3] = -inf
    L.down_dense[0, 40, 7] = inf
    L.down_dense[0, 40, 100] = inf
    y = moe.layer_forward_few(L, x, out_dtype=out)
    want = clean.double()
    want[:, 5] = h[:, 77].sign() * inf
    want[:, 130] = h[:, 3].sign() * -inf
    a, b = h[:, 7].sign() * inf, h[:, 100].sign() * inf
    want[:, 40] = a + b
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    fin = ~torch.isnan(want)
    assert torch.equal(y.double()[fin], want[fin])
