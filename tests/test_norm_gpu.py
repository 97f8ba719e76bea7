"""The norms between two blocks (moe_norm_forward) against 64 bits."""
import itertools

import pytest
import torch

import activation_sparse_expert_amd as moe
from dense_helpers import check, half_step
from gpu_helpers import DEV, Guarded, say
from rows_helpers import norm64, u

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.int8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)

    def __call__(self, shape, dt, std=1.0, at=0.0):
        return (torch.randn(shape, generator=self.g, device=DEV) * std + at).to(DT.get(dt, dt))


def make(n, d, wdt="f32", bias=False, post=False, offset=False, **kw):
    at = 0.0 if offset else 1.0
    return moe.Norm(d, w=n((d,), wdt, 0.3, at), b=n((d,), wdt, 0.3) if bias else None, post=post,
                    post_w=n((d,), wdt, 0.3, at) if post else None, post_b=n((d,), wdt, 0.3) if post and bias else None,
                    offset=offset, **kw)


def compare(norm, r, o, g, y, out, scale, what):
    v, ev, n, en = norm64(norm, r, o, g)
    if y is not None:
        check(y, v, ev + half_step(v.abs() + ev, y.dtype), what + " y")
    if out is None:
        return
    if out.dtype != torch.int8:
        check(out, n, en + half_step(n.abs() + en, out.dtype), what + " out")
        return
    top = n.abs().amax(1)
    check(scale, top / 127, (en.amax(1) + 2 * u * top) / 127 + 2.0 ** -149, what + " scale")
    # half a step of the code, the values' own bound, and the scale's share of 127 steps
    bound = en + (en.amax(1, keepdim=True) + 4 * u * top[:, None]) + (0.5 + 2.0 ** -12) * top[:, None] / 127
    check(out.double() * scale.double()[:, None], n, bound, what + " codes")
    assert bool((out.abs().amax(1) == 127).logical_or(scale == 0).all()), what + ": a row's largest code is 127"


# d on both sides of a lane's 8 values, of part and whole waves, of 2048, 4096, 8192 and 16384
SIZES = [(1, 1), (5, 2), (3, 7), (300, 8), (70, 63), (9, 64), (257, 100), (1000, 128), (33, 129), (65, 256), (6, 511), (7, 512),
         (12, 520), (5, 1000), (77, 1411), (3, 2048), (4, 2056), (2, 4096), (1, 4096), (3, 5000), (5, 6144), (2, 8192),
         (2, 8200), (3, 16383), (1, 16384), (2, 16384), (70000, 16)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,d", SIZES)
def test_against_64_bits(T, d, kind):
    cases = [dict(h="f16", o=None, out="f16", w="f16"), dict(h="bf16", o="bf16", out="bf16", w="bf16", post=True, offset=True),
             dict(h="f32", o="f16", out="f32", w="f32", gate="token", bias=True),
             dict(h="bf16", o="f32", out="i8", w="f32", gate="channel", bias=True, post=True, residual_scale=0.5, block_scale=2.0),
             dict(h="f32", o="bf16", out="i8", w="bf16", gate="channel", block_scale=0.25),
             dict(h=None, o="f16", out="f16", w="f32", post=True, bias=True, gate="token")]
    for i, c in enumerate(cases):
        c = dict(c)
        say(f"norm T={T} d={d} {kind} {c}")
        n = Draw(1000 * i + T + d)
        h, ot, out, gate = c.pop("h"), c.pop("o"), c.pop("out"), c.pop("gate", None)
        norm = make(n, d, c.pop("w"), kind=kind, eps=1e-5, **c)
        r = n((T, d), h, 2.0, 0.5) if h else None
        o = n((T, d), ot, 1.0, -0.25) if ot else None
        g = n((d,) if gate == "channel" else (T, d), ot) if gate else None
        y = Guarded((T, d), DT[h or ot]) if o is not None else None
        res, sc = Guarded((T, d), DT[out]), Guarded((T,), torch.float32)
        yy, nn, ss = moe.norm_forward(norm, r, o, gate=g, y=y.t if y else None, out=res.t,
                                      out_scale=sc.t if out == "i8" else None)
        torch.cuda.synchronize()
        for b, name in ((y, "y"), (res, "out"), (sc, "scale")):
            if b:
                b.check(name)
        compare(norm, r, o, g, yy, nn, ss, f"T={T} d={d} {kind} case {i}")
        again = moe.norm_forward(norm, r, o, gate=g, out_dtype=DT[out])
        assert torch.equal(nn, again[1]) and (y is None or torch.equal(yy, again[0])), "two runs differ"


@pytest.mark.parametrize("h,o,out", itertools.product(["f16", "bf16", "f32"], ["f16", "bf16", "f32"], DT))
@pytest.mark.parametrize("d", [96, 131])
def test_every_type(h, o, out, d):
    n = Draw(d)
    for w, gate in (("f16", None), ("bf16", "channel"), ("f32", "token")):
        norm = make(n, d, w, bias=True, post=w == "f32", kind="layer" if w == "bf16" else "rms")
        r, b = n((19, d), h, 1.5), n((19, d), o)
        g = n((d,) if gate == "channel" else (19, d), o) if gate else None
        compare(norm, r, b, g, *moe.norm_forward(norm, r, b, gate=g, out_dtype=DT[out]), f"{h} {o} {out} {w}")


@pytest.mark.parametrize("T,d", [(1, 48), (6, 64), (5, 1003), (3, 4096), (40, 128)])
def test_row_strides_and_in_place(T, d):
    """Column ranges of wider matrices, aligned and not; the columns between them stay; the residual is y."""
    for off, wide in ((8, d + 24), (3, d + 7)):
        n = Draw(T + d + off)
        norm = make(n, d, "f16", bias=True, post=True)
        stream = n((T, wide), "f16", 2.0)
        before = stream.clone()
        o, g = n((T, 2 * wide), "f16")[:, off:off + d], n((T, wide), "f16")[:, off:off + d]
        wide_out = torch.full((T, wide), 7.0, dtype=torch.float16, device=DEV)
        r = stream[:, off:off + d]
        y, out, _ = moe.norm_forward(norm, r, o, gate=g, y=r, out=wide_out[:, off:off + d])
        compare(norm, before[:, off:off + d], o, g, y, out, None, f"T={T} d={d}")
        for a, b in ((stream, before), (wide_out, torch.full_like(wide_out, 7.0))):
            assert torch.equal(a[:, :off], b[:, :off]) and torch.equal(a[:, off + d:], b[:, off + d:])


def test_what_is_not_wanted_is_not_written():
    n = Draw(4)
    norm = make(n, 200, "f32")
    r, o = n((9, 200), "f16"), n((9, 200), "f16")
    full = moe.norm_forward(norm, r, o)
    y, out, s = moe.norm_forward(norm, r, o, y=False)
    assert y is None and s is None and torch.equal(out, full[1])
    y, out, _ = moe.norm_forward(norm, r, o, out=False)
    assert out is None and torch.equal(y, full[0])
    y, out, _ = moe.norm_forward(norm, r)
    assert y is None and out.dtype == torch.float16
    y2 = torch.empty_like(r)
    moe.norm_forward(moe.Norm(200, residual_scale=0.5), r, y=y2, out=False)
    assert torch.equal(y2, r * 0.5)
    plain = moe.norm_forward(moe.Norm(200, kind="layer"), r, out_dtype=torch.float32)[1]
    compare(moe.Norm(200, kind="layer"), r, None, None, None, plain, None, "no weights")


@pytest.mark.parametrize("d", [16, 300, 4096, 9001])
def test_infinities_and_nan_stay_in_their_row(d):
    n = Draw(d)
    norm = make(n, d, "f32", post=True)
    r, o = n((7, d), "bf16"), n((7, d), "bf16")
    clean = moe.norm_forward(norm, r, o, out_dtype=torch.int8)
    r[1, d - 1] = float("nan")
    o[3, 0] = float("inf")
    r[5, d // 2] = float("-inf")
    y, q, s = moe.norm_forward(norm, r, o, out_dtype=torch.int8)
    good = [0, 2, 4, 6]
    for a, b in zip((y, q, s), clean):
        assert torch.equal(a[good], b[good])
    assert bool(torch.isnan(s[[1, 3, 5]]).all()) and not bool(q[[1, 3, 5]].any())
    out = moe.norm_forward(norm, r, o, out_dtype=torch.float32)[1]
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(out[3]).any()) and bool(torch.isnan(out[5, d // 2]))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [8, 1000, 7001])
def test_rows_from_the_smallest_to_the_largest(d, dt, kind):
    """Squares and sums that pass fp32, rows of zeros and of constants, rows that eps decides."""
    n = Draw(d)
    for scale in (1e37, 1e25, 1e18, 1.0, 1e-3, 1e-20, 1e-38, 0.0):
        r = n((5, d), "f32").mul(scale).clamp(-3e38, 3e38).to(DT[dt])
        norm = make(n, d, "f32", kind=kind, eps=1e-12)
        out = moe.norm_forward(norm, r, out_dtype=torch.float32)[1]
        compare(norm, r, None, None, None, out, None, f"{scale}")
    # (of equal values v - mean is what the mean's rounding leaves, which the bound has)
    r = torch.full((3, d), 5.0, dtype=DT[dt], device=DEV)
    norm = make(n, d, "f32", kind=kind)
    compare(norm, r, None, None, None, moe.norm_forward(norm, r, out_dtype=torch.float32)[1], None, "constant")
    out = moe.norm_forward(moe.Norm(d, kind=kind), torch.zeros((3, d), dtype=DT[dt], device=DEV), out_dtype=torch.int8)
    assert not bool(out[1].any()) and not bool(out[2].any())


def test_far_offsets():
    """Rows past 2^32 bytes in every operand."""
    T, d, stride = 17000, 72, 131072
    n = Draw(6)
    buf = torch.empty(T * stride, dtype=torch.float16, device=DEV).view(T, stride)
    r, o, g, out = (buf[:, 1024 * i:1024 * i + d] for i in range(4))
    for t in (r, o, g):
        t.copy_(n((T, d), "f16"))
    before = r.clone()
    norm = make(n, d, "f16", post=True)
    y, out, _ = moe.norm_forward(norm, r, o, gate=g, y=r, out=out)
    compare(norm, before, o, g, y, out, None, "far")


def test_many_short_rows():
    n = Draw(7)
    r = n((300000, 8), "bf16")
    norm = make(n, 8, "bf16")
    compare(norm, r, None, None, None, moe.norm_forward(norm, r)[1], None, "300000 x 8")


def test_graph_replays_and_streams():
    n = Draw(8)
    T, d = 33, 1000
    norm = make(n, d, "bf16", post=True)
    h, o = n((T, d), "f32"), n((T, d), "bf16")
    y, q, s = torch.empty_like(h), torch.empty((T, d), dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    moe.norm_forward(norm, h, o, y=y, out=q, out_scale=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.norm_forward(norm, h, o, y=y, out=q, out_scale=s)
    for i in range(4):
        h.copy_(n((T, d), "f32"))
        o.copy_(n((T, d), "bf16"))
        eager = moe.norm_forward(norm, h, o, out_dtype=torch.int8)
        for t in (y, q, s):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, q, s), eager)), f"replay {i}"
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        h2 = n((T, d), "f32")
        other = moe.norm_forward(norm, h2, o, out_dtype=torch.float32)[1]
    stream.synchronize()
    assert torch.equal(other, moe.norm_forward(norm, h2, o, out_dtype=torch.float32)[1])
