"""The linear layer (moe_linear_forward) against 64 bits."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from dense_helpers import check, linear64
from gpu_helpers import DEV, Guarded, say

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, shape, std, dt):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)


def layer(g, n, k, dt, gated=False, bias=False, act="none"):
    return moe.Linear(normal(g, (n, k), k ** -0.5, dt),
                      bias=normal(g, (n,), 0.5, torch.float32) if bias else None,
                      w_gate=normal(g, (n, k), k ** -0.5, dt) if gated else None,
                      bias_gate=normal(g, (n,), 0.5, torch.float32) if gated and bias else None, act=act)


def want(lin, x, residual, out):
    return linear64(x, lin.w, lin.bias, lin.w_gate, lin.bias_gate, lin.act, residual, out)


# T on both sides of 16, 32 and the tile sizes, k on both sides of 32, 64 and a
# batch of steps (256), n on both sides of 16, 64 and 128
SIZES = [(1, 8, 1), (1, 256, 704), (2, 40, 17), (16, 2056, 15), (17, 264, 33), (32, 1000, 129), (5, 4096, 1411),
         (33, 8, 1), (33, 72, 65), (64, 256, 64), (65, 1032, 127), (100, 2056, 1411), (128, 512, 128),
         (129, 64, 257), (257, 136, 300), (300, 4096, 512), (1000, 520, 1000), (2050, 72, 2049),
         (3000, 8, 4207), (3000, 200, 4208), (2900, 1000, 4207),
         (20, 4096, 1411), (24, 2056, 4000), (30, 2056, 16500), (24, 2056, 16400), (96, 1024, 512), (2, 16384, 40)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,k,n", SIZES)
def test_against_64_bits(T, k, n, dt):
    for i, (gated, bias, res, act, out) in enumerate([
            (False, False, False, "none", "f32"), (False, True, True, "gelu", dt),
            (True, True, True, "silu", dt), (True, False, False, "gelu_tanh", "f32"), (False, True, False, "relu", dt)]):
        say(f"linear T={T} k={k} n={n} {dt} gated={gated} {act} -> {out}")
        g = gen(1000 * i + T + k + n)
        lin = layer(g, n, k, DT[dt], gated, bias, act)
        x = normal(g, (T, k), 1.0, DT[dt])
        r = normal(g, (T, n), 1.0, DT[out]) if res else None
        y = Guarded((T, n), DT[out])
        ws = Guarded((moe.workspace_size(moe.OP_LINEAR, T, k, n),), torch.uint8)
        moe.linear_forward(lin, x, residual=r, y=y.t, ws=ws.t)
        again = moe.linear_forward(lin, x, residual=r, out_dtype=DT[out])
        torch.cuda.synchronize()
        y.check("y")
        ws.check("workspace")
        check(y.t, *want(lin, x, r, DT[out]), f"T={T} k={k} n={n}")
        assert torch.equal(y.t, again), "two runs differ"


@pytest.mark.parametrize("T", [1, 7, 31, 40, 200])
def test_row_strides_and_in_place(T):
    """x, y and the residual as column ranges of wider matrices; the columns
    between them stay as they were; the residual may be y."""
    g = gen(7 + T)
    k, n = 136, 75
    lin = layer(g, n, k, torch.float16, bias=True, act="silu")
    x = normal(g, (T, 3 * k), 1.0, torch.float16)[:, k:2 * k]
    wide = normal(g, (T, 200), 1.0, torch.float16)
    before = wide.clone()
    y = wide[:, 60:60 + n]
    moe.linear_forward(lin, x, residual=y, y=y)
    torch.cuda.synchronize()
    check(y, *want(lin, x, before[:, 60:60 + n], torch.float16), f"T={T}")
    assert torch.equal(wide[:, :60], before[:, :60]) and torch.equal(wide[:, 60 + n:], before[:, 60 + n:])


@pytest.mark.parametrize("T", [3, 50])
def test_infinities_and_nan_stay_in_their_row_and_column(T):
    """A NaN in one token or an infinity in one output's weights, k not a
    multiple of the tile: everything else is as without them."""
    g = gen(11)
    k, n = 104, 90
    lin = layer(g, n, k, torch.bfloat16)
    x = normal(g, (T, k), 1.0, torch.bfloat16)
    clean = moe.linear_forward(lin, x)
    x[1, k - 1] = float("nan")
    lin.w[n - 1, 0] = float("inf")
    y = moe.linear_forward(lin, x)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[1]).all())
    rows = [t for t in range(T) if t != 1]
    assert torch.equal(y[rows, :n - 1], clean[rows, :n - 1])
    assert bool(torch.isinf(y[rows, n - 1]).all())


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_activations_over_the_range(act, dt):
    """Arguments from -200 to 200 through an identity of weights, and a NaN."""
    k = 64
    lin = moe.Linear(torch.eye(k, device=DEV).to(DT[dt]), act=act)
    x = torch.linspace(-200, 200, 40 * k, device=DEV).view(40, k).to(DT[dt])
    x[0, 0] = float("nan")
    y = moe.linear_forward(lin, x)
    assert bool(torch.isnan(y[0, 0]))
    x[0, 0] = 0
    # a token's NaN reaches its whole row: take the rows without one
    check(y[1:], *want(lin, x[1:], None, torch.float32), act)


@pytest.mark.parametrize("T", [4, 48, 300])
def test_graph_replays_follow_their_inputs(T):
    g = gen(21)
    k, n = 1024, 512
    lin = layer(g, n, k, torch.bfloat16, gated=True, act="silu", bias=True)
    x = normal(g, (T, k), 1.0, torch.bfloat16)
    y = torch.empty((T, n), dtype=torch.bfloat16, device=DEV)
    ws = moe.new_workspace(moe.workspace_size(moe.OP_LINEAR, T, k, n))
    moe.linear_forward(lin, x, y=y, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.linear_forward(lin, x, y=y, ws=ws)
    for i in range(4):
        x.copy_(normal(g, (T, k), 1.0, torch.bfloat16))
        eager = moe.linear_forward(lin, x, out_dtype=torch.bfloat16)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager), f"replay {i}"


def test_two_streams_with_their_own_workspaces():
    g = gen(31)
    lin = layer(g, 700, 2048, torch.float16, bias=True, act="gelu")
    xs = [normal(g, (T, 2048), 1.0, torch.float16) for T in (60, 70)]
    alone = [moe.linear_forward(lin, x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    out = [None, None]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            for _ in range(5):
                out[i] = moe.linear_forward(lin, xs[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, out))


def test_far_offsets():
    """Rows past 2^32 bytes: 20000 tokens at a stride of 131072 elements."""
    g = gen(41)
    T, k, n, stride = 20000, 64, 40, 131072
    lin = layer(g, n, k, torch.float16)
    big = torch.empty(T * stride, dtype=torch.float16, device=DEV)
    x = big.view(T, stride)[:, :k]
    x.copy_(normal(g, (T, k), 1.0, torch.float16))
    y = big.view(T, stride)[:, 1024:1024 + n]
    moe.linear_forward(lin, x, y=y)
    check(y, *want(lin, x, None, torch.float16), "far")


@pytest.mark.parametrize("stride", [2 ** 21, 2 ** 21 + 8])
def test_rows_far_apart(stride):
    """Both sides of the stride up to which the offsets of a tile's rows have 32 bits."""
    g = gen(43)
    T, k, n = 40, 72, 4112
    lin = layer(g, n, k, torch.bfloat16, gated=True, act="silu")
    x = torch.empty(T * stride, dtype=torch.bfloat16, device=DEV).view(T, stride)[:, :k]
    x.copy_(normal(g, (T, k), 1.0, torch.bfloat16))
    check(moe.linear_forward(lin, x), *want(lin, x, None, torch.float32), "far rows")


@pytest.mark.parametrize("T,k,n", [(33000, 2048, 1), (33000, 4096, 40), (65536, 72, 24)])
def test_many_tokens(T, k, n):
    """The most tokens, and many whose products are split over K and joined."""
    g = gen(47)
    assert (moe.workspace_size(moe.OP_LINEAR, T, k, n) > 0) == (k > 72)
    lin = layer(g, n, k, torch.bfloat16, gated=True, bias=True, act="silu")
    x = normal(g, (T, k), 1.0, torch.bfloat16)
    check(moe.linear_forward(lin, x), *want(lin, x, None, torch.float32), f"T={T}")
