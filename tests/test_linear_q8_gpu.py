"""The linear layer on 8-bit integers (moe_linear_q8_forward) against 64 bits."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from dense_helpers import check
from gpu_helpers import DEV, Guarded, say
from rows_helpers import codes64, linear_q8_64

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.int8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, shape, dt, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)


def random_codes(g, shape):
    """Every code there is, -128 among them."""
    return torch.randint(-128, 128, shape, generator=g, device=DEV, dtype=torch.int8)


def layer(g, n, k, gated=False, bias=False, act="none"):
    def scales():
        return (torch.rand(n, generator=g, device=DEV) + 0.5) * (k ** -0.5 / 74)

    return moe.LinearQ8(random_codes(g, (n, k)), scales(), bias=normal(g, (n,), torch.float32, 0.5) if bias else None,
                        w_gate=random_codes(g, (n, k)) if gated else None, gate_scale=scales() if gated else None,
                        bias_gate=normal(g, (n,), torch.float32, 0.5) if gated and bias else None, act=act)


def tokens(g, T, k, kind):
    """(x, x_scale as the call takes them, the codes and scales that they stand for)"""
    if kind == "i8":
        q, s = random_codes(g, (T, k)), (torch.rand(T, generator=g, device=DEV) + 0.5) / 74
        return q, s, q, s
    x = normal(g, (T, k), DT[kind])
    return (x, None, *codes64(x))


# T on both sides of 1, 8, 16, 32 and the tile sizes, k on both sides of 64 and 128 and
# of a few blocks of those, n on both sides of 16, 64, 128 and 256
SIZES = [(1, 16, 1), (1, 256, 704), (1, 4096, 2100), (2, 48, 17), (7, 2064, 15), (8, 128, 129), (9, 272, 33), (16, 4112, 300),
         (17, 1040, 127), (24, 2064, 4000), (31, 144, 65), (32, 8208, 40), (30, 2064, 16500), (33, 16, 1), (33, 80, 65),
         (64, 256, 64), (65, 1040, 127), (96, 2048, 512), (100, 2064, 1411), (128, 512, 128), (129, 64, 257), (257, 144, 300),
         (300, 4096, 512), (1000, 528, 1000), (2050, 80, 2049), (3000, 16, 4207), (2900, 1008, 4207), (2, 65536, 40), (40, 131056, 24)]


@pytest.mark.parametrize("T,k,n", SIZES)
def test_against_64_bits(T, k, n):
    for i, (kind, gated, bias, res, act, out) in enumerate([
            ("i8", False, False, False, "none", "f32"), ("f16", False, True, True, "gelu", "f16"),
            ("i8", True, True, True, "silu", "bf16"), ("bf16", True, False, False, "gelu_tanh", "f32"),
            ("f32", False, True, False, "relu", "bf16")]):
        say(f"linear q8 T={T} k={k} n={n} {kind} gated={gated} {act} -> {out}")
        g = gen(1000 * i + T + k + n)
        lin = layer(g, n, k, gated, bias, act)
        x, sx, q, s = tokens(g, T, k, kind)
        r = normal(g, (T, n), DT[out]) if res else None
        y = Guarded((T, n), DT[out])
        ws = Guarded((moe.workspace_size(moe.OP_LINEAR_Q8, T, k, n, moe._row_dt(x), 0, 0),), torch.uint8)
        moe.linear_q8_forward(lin, x, x_scale=sx, residual=r, y=y.t, ws=ws.t)
        again = moe.linear_q8_forward(lin, x, x_scale=sx, residual=r, out_dtype=DT[out])
        torch.cuda.synchronize()
        y.check("y")
        ws.check("workspace")
        check(y.t, *linear_q8_64(q, s, lin, r, DT[out]), f"T={T} k={k} n={n} {kind}")
        assert torch.equal(y.t, again), "two runs differ"
        if kind != "i8":        # the call's own codes are quantize_rows'
            given = moe.linear_q8_forward(lin, q, x_scale=s, residual=r, out_dtype=DT[out])
            assert torch.equal(y.t, given), "codes made in the call and given"


@pytest.mark.parametrize("T", [1, 5, 20, 50, 300])
def test_sums_at_the_limits_of_32_bits(T):
    """All codes -128 over the longest k: 2^31 - 2^18 a sum, exact."""
    k, n = 131056, 18
    x = torch.full((T, k), -128, dtype=torch.int8, device=DEV)
    w = torch.full((n, k), -128, dtype=torch.int8, device=DEV)
    w[1] = 127
    one = torch.ones(max(T, n), device=DEV)
    y = moe.linear_q8_forward(moe.LinearQ8(w, one[:n].contiguous()), x, x_scale=one[:T].contiguous())
    want = torch.full((T, n), 128.0 * 128 * k, device=DEV, dtype=torch.float64)
    want[:, 1] = -128.0 * 127 * k
    assert torch.equal(y, want.float())


@pytest.mark.parametrize("kind", ["i8", "f16", "f32"])
@pytest.mark.parametrize("T", [1, 7, 31, 40, 200])
def test_row_strides_and_in_place(T, kind):
    """x, y and the residual as column ranges of wider matrices; the columns
    between them stay as they were; the residual may be y."""
    g = gen(7 + T)
    k, n = 144, 75
    lin = layer(g, n, k, bias=True, act="silu")
    x, sx, q, s = tokens(g, T, 3 * k, kind)
    x = x[:, k:2 * k]
    if kind == "i8":
        q = x
    else:
        q, s = codes64(x)
    wide = normal(g, (T, 200), torch.float16)
    before = wide.clone()
    y = wide[:, 60:60 + n]
    moe.linear_q8_forward(lin, x, x_scale=sx, residual=y, y=y)
    check(y, *linear_q8_64(q, s, lin, before[:, 60:60 + n], torch.float16), f"T={T}")
    assert torch.equal(wide[:, :60], before[:, :60]) and torch.equal(wide[:, 60 + n:], before[:, 60 + n:])


@pytest.mark.parametrize("T", [3, 50, 300])
def test_infinities_and_nan_stay_in_their_row_and_column(T):
    g = gen(11)
    k, n = 112, 90
    lin = layer(g, n, k)
    x = normal(g, (T, k), torch.bfloat16)
    x[2] = 0                                            # a row of zeros: scale 0
    clean = moe.linear_q8_forward(lin, x)
    assert not bool(clean[2].any())
    x[1, k - 1] = float("nan")
    x[0, 0] = float("inf")
    lin.w_scale[n - 1] = float("inf")
    y = moe.linear_q8_forward(lin, x)
    assert bool(torch.isnan(y[:2]).all())
    assert torch.equal(y[2:, :n - 1], clean[2:, :n - 1])
    assert not bool(torch.isfinite(y[3:, n - 1]).any())


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("k", [16, 128, 1040, 10240, 14336, 20480, 32768])
def test_one_token_of_any_length(k, kind):
    """Codes made by the product's own workgroups or, of long tokens, before it: the same outputs; rows
    of zeros, with a NaN, an infinity, and of the smallest and largest numbers."""
    g = gen(k)
    fi = torch.finfo(DT[kind])
    for n, gated in ((17, False), (300, True), (9000, False)):
        lin = layer(g, n, k, gated, True, "silu")
        base = normal(g, (1, k), DT[kind])
        for change in (None, 0.0, float("nan"), float("inf"), fi.max, fi.smallest_normal * fi.eps):
            x = base.clone()
            if change == 0.0 or (change is not None and change == change and change < 1):
                x.zero_()
            if change is not None:
                x[0, k - 1] = change
            q, s = codes64(x)
            y = moe.linear_q8_forward(lin, x)
            # (a row with an infinity or a NaN has the scale NaN)
            assert torch.equal(y.isnan(), ~s.isfinite()[:, None].expand_as(y)), f"{n} {change}"
            given = moe.linear_q8_forward(lin, *moe.quantize_rows(x)[:1], x_scale=moe.quantize_rows(x)[1])
            assert bool(((y == given) | (y.isnan() & given.isnan())).all()), f"{n} {change}"
            if change is None:
                check(y, *linear_q8_64(q, s, lin), f"{n}")


@pytest.mark.parametrize("T", [1, 20, 48, 300])
def test_graph_replays_follow_their_inputs(T):
    """Two graphs on one workspace, replayed in turn with eager work between."""
    g = gen(21)
    k, n = 1024, 512
    lin = layer(g, n, k, gated=True, act="silu", bias=True)
    xs = [normal(g, (T, k), torch.bfloat16) for _ in range(2)]
    ys = [torch.empty((T, n), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    ws = moe.new_workspace(moe.workspace_size(moe.OP_LINEAR_Q8, T, k, n, moe.MOE_BF16, 0, 0))
    graphs = []
    for x, y in zip(xs, ys):
        moe.linear_q8_forward(lin, x, y=y, ws=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            moe.linear_q8_forward(lin, x, y=y, ws=ws)
    for i in range(4):
        for x, y in zip(xs, ys):
            x.copy_(normal(g, (T, k), torch.bfloat16))
            y.zero_()
        eager = [moe.linear_q8_forward(lin, x, out_dtype=torch.bfloat16) for x in xs]
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, e) for y, e in zip(ys, eager)), f"replay {i}"


def test_two_streams_with_their_own_workspaces():
    g = gen(31)
    lin = layer(g, 700, 2048, bias=True, act="gelu")
    xs = [normal(g, (T, 2048), torch.float16) for T in (60, 70)]
    alone = [moe.linear_q8_forward(lin, x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    out = [None, None]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            for _ in range(5):
                out[i] = moe.linear_q8_forward(lin, xs[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, out))


@pytest.mark.parametrize("T,stride", [(20000, 262144), (40, 1 << 21), (40, (1 << 22) + 16), (40, 1 << 23)])
def test_far_offsets(T, stride):
    """Rows past 2^32 bytes, and rows far apart in one tile."""
    g = gen(41)
    k, n = 80, 40 if T > 1000 else 4112
    lin = layer(g, n, k, gated=True, act="silu")
    buf = torch.empty(T * stride, dtype=torch.int8, device=DEV).view(T, stride)
    x = buf[:, :k]
    x.copy_(random_codes(g, (T, k)))
    s = torch.rand(T, generator=g, device=DEV) + 0.5
    y = buf.view(torch.float16)[:, 1024:1024 + n]
    moe.linear_q8_forward(lin, x, x_scale=s / 74, y=y)
    check(y, *linear_q8_64(x, s / 74, lin, None, torch.float16), "far")


@pytest.mark.parametrize("T,k,n", [(33000, 2048, 1), (33000, 4096, 40), (65536, 80, 24)])
def test_many_tokens(T, k, n):
    g = gen(47)
    lin = layer(g, n, k, gated=True, bias=True, act="silu")
    x = random_codes(g, (T, k))
    s = (torch.rand(T, generator=g, device=DEV) + 0.5) / 74
    check(moe.linear_q8_forward(lin, x, x_scale=s), *linear_q8_64(x, s, lin), f"T={T}")


def test_a_decode_step():
    """Norm to codes, gated 8-bit product, down product into the stream, norm, few-token MoE layer: each call
    against its own 64-bit form, then the run of them captured and replayed."""
    from test_few_gpu import make
    g = gen(61)
    T, d, f = 6, 512, 1408
    h0 = normal(g, (T, d), torch.bfloat16)
    block = normal(g, (T, d), torch.bfloat16)
    one = moe.Norm(d, w=normal(g, (d,), torch.bfloat16, 0.2), offset=True)
    two = moe.Norm(d, kind="layer", w=normal(g, (d,), torch.bfloat16, 0.2), offset=True, post=True, residual_scale=0.5)
    up = moe.LinearQ8(*moe.quantize_rows(normal(g, (f, d), torch.bfloat16, d ** -0.5)), act="silu")
    up.w_gate, up.gate_scale = moe.quantize_rows(normal(g, (f, d), torch.bfloat16, d ** -0.5))
    down = moe.LinearQ8(*moe.quantize_rows(normal(g, (d, f), torch.bfloat16, f ** -0.5)))
    few = make(g, d, 256, 8, 2, 1, torch.bfloat16)

    def step(h):
        h, q, s = moe.norm_forward(one, h, block, y=h, out_dtype=torch.int8)
        a = moe.linear_q8_forward(up, q, x_scale=s, out_dtype=torch.bfloat16)
        b = moe.linear_q8_forward(down, a, residual=h, out_dtype=torch.bfloat16)
        h2, n, _ = moe.norm_forward(two, h, b, out_dtype=torch.bfloat16)
        return q, s, a, b, h2, n, moe.layer_forward_few(few, n, residual=h2, out_dtype=torch.bfloat16)

    h = h0.clone()
    q, s, a, b, h2, n, y = step(h)
    from test_norm_gpu import compare
    compare(one, h0, block, None, h, q, s, "norm to codes")
    check(a, *linear_q8_64(q, s, up, None, torch.bfloat16), "gated")
    check(b, *linear_q8_64(*codes64(a), down, h, torch.bfloat16), "down")
    compare(two, h, b, None, h2, n, None, "norm")
    hs = h0.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(hs)
    for i in range(3):
        hs.copy_(normal(g, (T, d), torch.bfloat16))
        want = step(hs.clone())
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, w) for p, w in zip(got, want)), f"replay {i}"
