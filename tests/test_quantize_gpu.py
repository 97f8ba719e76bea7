"""Rows to 8-bit codes and back (moe_quantize_rows, moe_dequantize_rows) against exact arithmetic."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from gpu_helpers import DEV, Guarded, say
from rows_helpers import codes64, u
from dense_helpers import check, half_step

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def normal(seed, shape, dt, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)


# k on both sides of a lane's 8 or 16 values, of a wave's, of a workgroup's and of what registers hold
SIZES = [(1, 1), (1, 7), (3, 8), (5, 15), (2, 16), (70, 63), (9, 64), (4, 127), (300, 128), (65, 255), (17, 513), (33, 1000),
         (6, 1024), (5, 1411), (7, 2048), (3, 4096), (2, 8190), (4, 8192), (1, 14336), (3, 16383), (2, 16384), (2, 16392),
         (2, 40000), (1, 131072), (70000, 24), (1, 1 << 20)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,k", SIZES)
def test_codes_and_values(T, k, dt):
    say(f"rows T={T} k={k} {dt}")
    x = normal(T + k, (T, k), DT[dt])
    q, s = Guarded((T, k), torch.int8), Guarded((T,), torch.float32)
    moe.quantize_rows(x, q=q.t, scale=s.t)
    torch.cuda.synchronize()
    q.check("q")
    s.check("scale")
    wq, ws = codes64(x)
    assert torch.equal(q.t, wq) and torch.equal(s.t, ws)
    for out in DT:
        y = Guarded((T, k), DT[out])
        moe.dequantize_rows(q.t, s.t, y=y.t)
        torch.cuda.synchronize()
        y.check("y")
        want = wq.double() * ws.double()[:, None]
        check(y.t, want, u * want.abs() + half_step(want, DT[out]), out)


@pytest.mark.parametrize("dt", DT)
def test_ties_go_to_even(dt):
    """Rows whose quotients are all n + 1/2: x = (2 n + 1) 2^e beside a largest value of 254 2^e."""
    x = (2 * torch.arange(-127, 127, device=DEV) + 1).double().clamp(-253, 253)
    x = torch.cat([torch.tensor([254.0], device=DEV, dtype=torch.float64), x])
    x = torch.stack([x * 2.0 ** e for e in ((-12, -6, 0, 5) if dt == "f16" else (-120, -30, 0, 40, 110))]).to(DT[dt])
    q, s = moe.quantize_rows(x)
    wq, ws = codes64(x)
    assert torch.equal(q, wq) and torch.equal(s, ws)


@pytest.mark.parametrize("dt", DT)
def test_every_16_bit_quotient(dt):
    """All significands of one binade beside largest values over the next two: every near-tie there is."""
    base = torch.arange(1024, 2048, device=DEV).float() / 1024
    tops = torch.arange(1024, 4096, 37, device=DEV).float() / 1024
    x = torch.cat([base.expand(len(tops), -1), 0.37 * base.expand(len(tops), -1), tops[:, None] + 1], 1).to(DT[dt])
    q, s = moe.quantize_rows(x)
    wq, ws = codes64(x)
    assert torch.equal(q, wq) and torch.equal(s, ws)


@pytest.mark.parametrize("dt", DT)
def test_the_smallest_and_largest_values(dt):
    fi = torch.finfo(DT[dt])
    tiny = fi.smallest_normal * fi.eps
    rows = [[fi.max, -fi.max, fi.max / 2, 1.0], [tiny, -tiny, 0.0, 0.0], [tiny * 100, tiny * 3, -tiny * 50, 0.0],
            [fi.smallest_normal, fi.smallest_normal / 2, 0.0, -fi.smallest_normal], [0.0, -0.0, 0.0, 0.0],
            [fi.max, fi.smallest_normal, tiny, 0.0], [1.0, -1.0, 0.5, -0.5]]
    x = torch.tensor(rows, dtype=torch.float64).to(DT[dt]).to(DEV)
    q, s = moe.quantize_rows(x)
    wq, ws = codes64(x)
    assert torch.equal(q, wq) and torch.equal(s, ws)
    y = moe.dequantize_rows(q, s, out_dtype=DT[dt])
    # fp32's largest value M: M / 127 rounds up to a scale with 127 scale >= 2^128 - 2^103, which fp32
    # rounds to infinity; every other row is finite
    assert torch.equal(y, (wq.float() * ws[:, None]).to(DT[dt])) and not bool(y[4].any())
    far = 127 * ws.double()[0] >= 2.0 ** 128 - 2.0 ** 103
    assert bool(far) == (dt == "f32") and bool(torch.isinf(y[0, 0])) == (dt == "f32")
    assert bool(torch.isfinite(y[[1, 2, 3, 4, 6]]).all())


@pytest.mark.parametrize("k", [5, 64, 700, 9000, 20000])
def test_infinities_and_nan_stay_in_their_row(k):
    x = normal(3, (7, k), torch.bfloat16)
    clean = moe.quantize_rows(x)
    x[1, k - 1] = float("nan")
    x[3, 0] = float("inf")
    x[5, k // 2] = float("-inf")
    x[5, 0] = float("nan")
    q, s = moe.quantize_rows(x)
    bad, good = [1, 3, 5], [0, 2, 4, 6]
    assert bool(torch.isnan(s[bad]).all()) and not bool(q[bad].any())
    assert torch.equal(q[good], clean[0][good]) and torch.equal(s[good], clean[1][good])
    assert bool(torch.isnan(moe.dequantize_rows(q, s)[bad]).all())


@pytest.mark.parametrize("T,k,wide", [(1, 40, 50), (5, 64, 96), (6, 130, 131), (40, 1000, 1003), (3, 9000, 9111)])
@pytest.mark.parametrize("dt", DT)
def test_row_strides(T, k, wide, dt):
    """Column ranges of wider matrices at odd offsets; the columns between them stay as they were."""
    x = normal(k, (T, 2 * wide), DT[dt])[:, 3:3 + k]
    q = torch.full((T, wide), 77, dtype=torch.int8, device=DEV)
    at = wide - k - 1 if wide - k > 1 else 0
    moe.quantize_rows(x, q=q[:, at:at + k])
    wq, ws = codes64(x)
    assert torch.equal(q[:, at:at + k], wq) and bool((q[:, :at] == 77).all()) and bool((q[:, at + k:] == 77).all())
    y = torch.full((T, wide + 5), 7.0, dtype=DT[dt], device=DEV)
    moe.dequantize_rows(q[:, at:at + k], ws, y=y[:, 1:1 + k])
    assert bool((y[:, 0] == 7).all()) and bool((y[:, 1 + k:] == 7).all())
    want = wq.double() * ws.double()[:, None]
    check(y[:, 1:1 + k], want, u * want.abs() + half_step(want, DT[dt]), "strided")


def test_far_offsets():
    """Rows past 2^32 bytes on both sides."""
    T, k, stride = 17000, 40, 262144
    buf = torch.empty(T * stride, dtype=torch.int8, device=DEV)
    x = buf.view(torch.float16).view(T, stride // 2)[:, :k]
    x.copy_(normal(5, (T, k), torch.float16))
    q = buf.view(T, stride)[:, 1024:1024 + k]
    _, s = moe.quantize_rows(x, q=q)
    wq, ws = codes64(x)
    assert torch.equal(q, wq) and torch.equal(s, ws)
    y = buf.view(torch.float16).view(T, stride // 2)[:, 4096:4096 + k]
    moe.dequantize_rows(q, s, y=y)
    assert torch.equal(y, (wq.float() * ws[:, None]).half())


def test_graph_replays_and_streams():
    x = normal(8, (33, 1000), torch.bfloat16)
    q, s = torch.empty((33, 1000), dtype=torch.int8, device=DEV), torch.empty(33, device=DEV)
    y = torch.empty((33, 1000), dtype=torch.bfloat16, device=DEV)
    moe.dequantize_rows(*moe.quantize_rows(x, q=q, scale=s), y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.dequantize_rows(*moe.quantize_rows(x, q=q, scale=s), y=y)
    for i in range(4):
        x.copy_(normal(20 + i, (33, 1000), torch.bfloat16))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        wq, ws = codes64(x)
        assert torch.equal(q, wq) and torch.equal(s, ws), f"replay {i}"
        assert torch.equal(y, (wq.float() * ws[:, None]).bfloat16())
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        x2 = normal(9, (33, 1000), torch.bfloat16)
        q2, s2 = moe.quantize_rows(x2)
    stream.synchronize()
    assert torch.equal(q2, codes64(x2)[0])
