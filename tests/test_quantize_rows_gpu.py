"""Rows to 8-bit codes and back, more rows than workgroups, against exact arithmetic."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from dense_helpers import check, half_step
from gpu_helpers import DEV, say
from rows_helpers import codes64, u
from test_quantize_gpu import DT, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


# Rows of part of a wave go in 4096 workgroups of 256 lanes (8 lanes up to 64 columns, 16 up to 128 and so on),
# others in workgroups of 2 to 16 waves, 24 waves on each of 256 compute units; the last two are read twice
SIZES = [(300011, 61), (280001, 64), (150001, 100), (70003, 203), (36007, 504), (33013, 512), (9001, 520), (6007, 1411),
         (5003, 2048), (3301, 4096), (3001, 5000), (2111, 8191), (1301, 12000), (1031, 16383), (1033, 16384), (700, 16391), (513, 20000)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,k", SIZES)
def test_more_rows_than_workgroups(T, k, dt):
    say(f"rows T={T} k={k} {dt}")
    x = normal(T + k, (T, k), DT[dt])
    x[T // 2] = 0
    x[T - 1, k - 1] = float("inf")
    q, s = moe.quantize_rows(x)
    x[T - 1] = 0
    wq, ws = codes64(x)
    assert torch.equal(q, wq) and torch.equal(s[:-1], ws[:-1]) and bool(torch.isnan(s[-1]))
    y = moe.dequantize_rows(q, s, out_dtype=DT[dt])
    want = wq[:-1].double() * ws[:-1].double()[:, None]
    check(y[:-1], want, u * want.abs() + half_step(want, DT[dt]), f"T={T} k={k} {dt}")
    assert bool(torch.isnan(y[-1]).all())


@pytest.mark.parametrize("k", [8, 520])
def test_more_than_a_million_rows(k):
    """Past the 2^20 workgroups of a grid, a row to each from 520 columns on."""
    T = (1 << 20) + 77 if k > 512 else (1 << 25) + 77
    q = torch.randint(-127, 128, (T, k), device=DEV, dtype=torch.int8)
    s = torch.rand(T, device=DEV) + 0.5
    y = moe.dequantize_rows(q, s, out_dtype=torch.bfloat16)
    q2, s2 = moe.quantize_rows(y)
    for at in range(0, T, 1 << 18 if k > 512 else 1 << 24):
        part = slice(at, min(T, at + (1 << 18 if k > 512 else 1 << 24)))
        assert torch.equal(y[part], (q[part].float() * s[part, None]).to(torch.bfloat16)), at
        wq, ws = codes64(y[part])
        assert torch.equal(q2[part], wq) and torch.equal(s2[part], ws), at


@pytest.mark.parametrize("e", [-140, -126, -100, -20, 0, 60, 126])
def test_32_bit_numbers_next_to_ties(e):
    """For 4096 largest values a 2^e: the fp32 numbers nearest to each (n + 1/2) a / 127, and their neighbours; where
    a is a multiple of 254 the ties themselves."""
    g = torch.Generator(device=DEV)
    g.manual_seed(e + 200)
    a = torch.randint(1 << 23, 1 << 24, (4096,), generator=g, device=DEV).double()
    a[::3] = 254 * torch.floor(a[::3] / 254)
    n = torch.arange(-127, 127, device=DEV).double()
    near = ((n + 0.5) * a[:, None] / 127).float()
    x = torch.cat([a.float()[:, None], near, torch.nextafter(near, torch.full_like(near, 1e30)),
                   torch.nextafter(near, torch.full_like(near, -1e30))], 1)
    x = (x.double() * 2.0 ** (e - 23)).float()          # (subnormals are rounded again)
    q, s = moe.quantize_rows(x)
    wq, ws = codes64(x)
    assert torch.equal(q, wq) and torch.equal(s, ws)
