"""The norms between two blocks where every value of a row is the same, however large, and where eps
counts beside squares that pass fp32."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from dense_helpers import check, half_step
from gpu_helpers import DEV
from rows_helpers import u
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


@pytest.mark.parametrize("with_block", [False, True])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d", [2, 3, 7, 63, 100, 255, 500, 1000, 2047, 2966, 5000, 7001, 12000, 16383])
def test_equal_values_of_any_size(d, dt, with_block):
    """A sum of d equal values is not exact in fp32, but it is off by few units in the last place, and so is the
    mean; v - mean then has at most 7 bits and its sum, with the 14 of d, is exact, and so is what the mean is off by."""
    values = [1.0, 1000.0, -30000.0, 0.1, 5.0, -1 / 3, 1e-3, 60000.0]
    if dt != "f16":
        values += [1e37, -3.3e38, 1e20, 1.7e38, 12345678.0, 1e-30]
    expect_bias_alone(d, rows(values, d, dt), with_block)


def centred64(z, eps):
    """(N(z), its bound) of a layer norm without weights, z exact.  The mean that fp32 makes is off by at most
    b = (chain + 2) u mean|z|; e = z - it is rounded once, the mean of e is off by (chain + 2) u mean|e|
    and the difference of both is rounded once.  Of the squares about the mean, sum e^2 is off by
    (chain + 4) u of itself, b^2 d of it at most being taken out again, and 1 / sqrt has half of that error and
    a few roundings of its own."""
    d = z.shape[1]
    chain = d / 64 + 16
    c = z - z.mean(1, keepdim=True)
    b = (chain + 2) * u * z.abs().mean(1, keepdim=True)
    mean_e = c.abs().mean(1, keepdim=True) + b
    ec = u * (c.abs() + b) + (chain + 3) * u * mean_e + u * c.abs()
    var = (c * c).mean(1, keepdim=True)
    f = 1 / torch.sqrt(var + eps)
    n = c * f
    rel = f * f * ((chain + 6) * u * (var + 2 * b * b) + (c.abs() * ec).mean(1, keepdim=True))
    return n, ec * f + n.abs() * (rel + 8 * u) + 2.0 ** -149


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,d", [(5, 7), (4, 100), (3, 1000), (3, 4096), (2, 7001), (2, 16384)])
def test_rows_far_from_zero(T, d, dt):
    """Values around an offset that is large beside their spread (in 16 bits: as far as the type holds a spread)."""
    n = Draw(d)
    # b below: at most 274 u of the offset; the spread stays 60 times that or more
    for at in (30.0, 1000.0) if dt != "f32" else (30.0, 1000.0, -1000.0):
        r = n((T, d), dt, at / 100 if dt == "bf16" else 1.0, at)
        out = moe.norm_forward(moe.Norm(d, kind="layer", eps=1e-6), r, out_dtype=torch.float32)[1]
        want, bound = centred64(r.double(), 1e-6)
        check(out, want, bound + half_step(want, torch.float32), f"T={T} d={d} {dt} at {at}")
