"""The linear layer's activations relative to their own value, where it is far
smaller than the argument.

x times an identity is exact, so y is the activation of x.  In u = 2^-24:
  gelu: erfc(a), a = -v / sqrt 2, with a rounded once and its constant once
    (1.5 u), is off by (2 a^2 + 1.5 |a|) 1.5 u <= (1.5 v^2 + 1.7 |v|) u, and by the 16
    units (32 u) that a library's erfc may be off; three products, the epilogue's rounding.
  silu: exp(-v) off by (2 |v| + 2) u, the sum by one, the reciprocal by two, the product by one.
  gelu_tanh: the same with z = 2 sqrt(2 / pi) (v + 0.044715 v^3) for v, which is itself
    off by 7 u.
Below 2^-126 nothing is asked."""
import math

import pytest
import torch

import activation_sparse_expert_amd as moe
from dense_helpers import act64
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def relative(v, act):
    if act == "gelu":
        return (1.5 * v * v + 1.7 * v.abs() + 38) * U
    if act == "silu":
        return (2 * v.abs() + 8) * U
    z = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3).abs()
    return (9 * z + 8) * U


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("T", [30, 4000])
def test_relative_to_the_value(act, dt, T):
    """30 tokens stream, 4000 go in tiles."""
    k = 64
    n = 64 if T < 100 else 2112
    lin = moe.Linear(torch.eye(k, device=DEV).repeat(n // k, 1).to(DT[dt]), act=act)
    x = torch.linspace(-9, 9, T * k, device=DEV).view(T, k).to(DT[dt])
    y = moe.linear_forward(lin, x)
    v = x.double().repeat(1, n // k)
    want = act64(v, act)
    bound = want.abs() * relative(v, act) + 2.0 ** -126
    e = (y.double() - want).abs()
    worst, within = int((e / bound).argmax()), bool((e <= bound).all())
    say(f"{act} {dt} T={T}: worst {float((e / bound).max()):.3g} bounds at {float(v.flatten()[worst])}")
    assert within
