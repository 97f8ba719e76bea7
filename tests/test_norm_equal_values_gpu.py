"""The norms between two blocks where every value of a row is the same, however large, and where eps
counts beside squares that pass fp32."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from gpu_helpers import DEV
from test_norm_gpu import DT, Draw, compare, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def rows(values, d, dt):
    return torch.tensor(values, dtype=torch.float64, device=DEV)[:, None].expand(-1, d).to(DT[dt]).contiguous()


def expect_bias_alone(d, r, with_block):
    """Layer norms of rows of equal values: v - mean is 0, so out is the bias (and a post norm adds its own)."""
    n = Draw(d)
    norm = make(n, d, "f32", bias=True, kind="layer", post=with_block)
    b, pb = norm.b, norm.post_b
    norm.b = norm.post_b = None
    zero = torch.zeros_like(r)
    for out in DT:
        if with_block:
            y, z, s = moe.norm_forward(norm, zero, r, out_dtype=DT[out])
            assert not bool(y.any()), f"{out} y"
        else:
            _, z, s = moe.norm_forward(norm, r, out_dtype=DT[out])
        assert not bool(z.any()) and (s is None or not bool(s.any())), f"{out} d={d}"
    norm.b, norm.post_b = b, pb
    y, z, _ = moe.norm_forward(norm, zero, r, out_dtype=DT["f32"]) if with_block else \
        moe.norm_forward(norm, r, out_dtype=DT["f32"])
    if with_block:
        assert torch.equal(y, pb.to(y.dtype).expand_as(y))
    else:
        assert torch.equal(z, b.expand_as(z))


@pytest.mark.parametrize("with_block", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [8, 64, 256, 2048, 16384])
def test_equal_values_whose_sum_passes_fp32(d, dt, with_block):
    """(powers of two and widths that are powers of two: every partial sum is exact until it overflows)"""
    top = 2.0 ** 127 / d
    expect_bias_alone(d, rows([2.0 ** 126, -2.0 ** 126, 2.0 ** 127, 2 * top, top, -4 * top, 1.0], d, dt), with_block)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [8, 100, 1000, 7001])
def test_a_large_eps_beside_squares_that_pass_fp32(d, dt, kind):
    n = Draw(d)
    for eps in (1e30, 1e36, 3e38):
        for std in (1e18, 2e19, 3e20, 1e25):
            r = n((5, d), "f32").mul(std).to(DT[dt])
            norm = make(n, d, "f32", kind=kind, eps=eps)
            out = moe.norm_forward(norm, r, out_dtype=torch.float32)[1]
            compare(norm, r, None, None, None, out, None, f"eps {eps} std {std}")
