"""The linear layer's tile kernels against 64 bits: every tile, plain and gated,
with and without a split of k; strides, special values, streams and graphs in
them (sizes that tests/test_linear_gpu.py streams past the tokens instead)."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from dense_helpers import check
from gpu_helpers import DEV, Guarded, say
from linear_sizes import TILES
from test_linear_gpu import DT, gen, layer, normal, want

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,k,n,tile,gated,split", TILES)
def test_every_tile_against_64_bits(T, k, n, tile, gated, split, dt):
    for act, out in (("silu" if gated else "gelu", dt), ("relu" if gated else "none", "f32")):
        say(f"linear T={T} k={k} n={n} {dt} tile {tile} gated={gated} split={split} {act} -> {out}")
        g = gen(T + k + n)
        lin = layer(g, n, k, DT[dt], gated, True, act)
        x, r = normal(g, (T, k), 1.0, DT[dt]), normal(g, (T, n), 1.0, DT[out])
        y = Guarded((T, n), DT[out])
        nbytes = moe.workspace_size(moe.OP_LINEAR, T, k, n)
        assert nbytes > 0 or not split
        ws = Guarded((max(nbytes, 16),), torch.uint8)
        moe.linear_forward(lin, x, residual=r, y=y.t, ws=ws.t)
        again = moe.linear_forward(lin, x, residual=r, out_dtype=DT[out])
        torch.cuda.synchronize()
        y.check("y")
        ws.check("workspace")
        check(y.t, *want(lin, x, r, DT[out]), f"T={T} k={k} n={n}")
        assert torch.equal(y.t, again), "two runs differ"


# (T, k, n, gated, split) with n a multiple of 4, so that outputs may go by fours: a
# small tile, a large one, and one of each whose split is joined
QUADS = [(36, 200, 2152, True, False), (276, 224, 11212, False, False), (67, 1368, 1364, True, True),
         (68, 2408, 4224, False, True)]


@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("T,k,n,gated,split", QUADS)
@pytest.mark.parametrize("left,stride", [(64, 128), (62, 128), (61, 128), (64, 129)])
def test_strides_and_in_place(T, k, n, gated, split, left, stride, out):
    """y and residual in one column range of a wider matrix, aligned for reads of four
    or not; the columns beside it stay as they were."""
    g = gen(T + n + left)
    lin = layer(g, n, k, torch.float16, gated, True, "silu")
    assert (moe.workspace_size(moe.OP_LINEAR, T, k, n) > 0) or not split
    x = normal(g, (T, 3 * k), 1.0, torch.float16)[:, k:2 * k]
    wide = normal(g, (T, n + stride), 1.0, DT[out])
    before = wide.clone()
    y = wide[:, left:left + n]
    moe.linear_forward(lin, x, residual=y, y=y)
    torch.cuda.synchronize()
    check(y, *want(lin, x, before[:, left:left + n], DT[out]), f"T={T} left={left}")
    assert torch.equal(wide[:, :left], before[:, :left]) and torch.equal(wide[:, left + n:], before[:, left + n:])


@pytest.mark.parametrize("T,k,n,gated,split", QUADS)
def test_special_values_stay_in_their_row_and_column(T, k, n, gated, split):
    """A NaN at the end of one token's row and an infinity in one output's weights,
    k not a multiple of 64: everything else is as without them."""
    g = gen(13 + T)
    lin = layer(g, n, k, torch.bfloat16, gated)
    x = normal(g, (T, k), 1.0, torch.bfloat16)
    clean = moe.linear_forward(lin, x)
    x[1, k - 1] = float("nan")
    x[T - 1, k - 8] = float("inf")
    lin.w[n - 1, 0] = float("inf")
    lin.w[7, k - 1] = float("nan")
    y = moe.linear_forward(lin, x)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[T - 1]).any())
    rows = [t for t in range(T) if t not in (1, T - 1)]
    cols = [c for c in range(n - 1) if c != 7]
    assert torch.equal(y[rows][:, cols], clean[rows][:, cols])
    assert bool(torch.isinf(y[rows, n - 1]).all()) and bool(torch.isnan(y[rows, 7]).all())


@pytest.mark.parametrize("T,k,n,gated,split", QUADS)
def test_graph_replays_follow_their_inputs(T, k, n, gated, split):
    g = gen(23)
    lin = layer(g, n, k, torch.bfloat16, gated, True, "silu")
    x = normal(g, (T, k), 1.0, torch.bfloat16)
    y = torch.empty((T, n), dtype=torch.bfloat16, device=DEV)
    ws = moe.new_workspace(moe.workspace_size(moe.OP_LINEAR, T, k, n))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.linear_forward(lin, x, y=y, ws=ws)
    for i in range(4):
        x.copy_(normal(g, (T, k), 1.0, torch.bfloat16))
        eager = moe.linear_forward(lin, x, out_dtype=torch.bfloat16)
        y.zero_()
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager), f"replay {i}"


def test_two_streams_with_their_own_workspaces():
    g = gen(33)
    n, k = 1362, 1368
    lin = layer(g, n, k, torch.float16, True, True, "silu")
    xs = [normal(g, (T, k), 1.0, torch.float16) for T in (67, 75)]
    assert all(moe.workspace_size(moe.OP_LINEAR, x.shape[0], k, n) > 0 for x in xs)
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
