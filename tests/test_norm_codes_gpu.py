"""A norm's codes are those that quantize_rows makes of its 32-bit output, to the last one."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from gpu_helpers import DEV
from rows_helpers import codes64
from test_norm_gpu import DT, Draw, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,d", [(130000, 40), (40000, 128), (20000, 500), (6000, 1411), (4000, 4096), (1500, 8192), (300, 16384)])
def test_codes_are_those_of_the_row_quantiser(T, d, kind):
    """(some million quotients: a rounding of 127 x to 24 bits moves several of them over a border)"""
    for i, (h, o, w) in enumerate((("bf16", "bf16", "bf16"), ("f32", "f16", "f32"))):
        n = Draw(10 * d + i)
        norm = make(n, d, w, bias=i == 1, post=True, kind=kind)
        r, b = n((T, d), h, 1.5), n((T, d), o)
        x = moe.norm_forward(norm, r, b, out_dtype=torch.float32)[1]
        _, q, s = moe.norm_forward(norm, r, b, out_dtype=torch.int8)
        want, scale = codes64(x)
        assert torch.equal(s, scale), f"{h} scales"
        off = q != want
        assert not bool(off.any()), f"{h} T={T} d={d}: {int(off.sum())} of {off.numel()} codes differ"
        again, _ = moe.quantize_rows(x)
        assert torch.equal(again, q)


def test_ties_go_to_even():
    """With w = 0 the norm is its bias: odd multiples of half a step of the largest value, exact and rounded to 24 bits."""
    b = torch.cat([torch.tensor([254.0]), 2 * torch.arange(-126, 126) + 1]).to(DEV)
    for scale in (1.0, 3.0, 1 / 7, 1e-20, 1e20):
        bias = (b * scale).contiguous()
        norm = moe.Norm(len(b), w=torch.zeros_like(b), b=bias)
        x = torch.ones((2, len(b)), device=DEV, dtype=DT["f16"])
        _, q, s = moe.norm_forward(norm, x, out_dtype=torch.int8)
        want, ws = codes64(bias.expand(2, -1))
        assert torch.equal(q, want) and torch.equal(s, ws), scale
