"""The tile kernels of the linear layer on 8-bit integers against 64 bits: every tile, plain
and gated, with and without a split of k; strides in them (sizes that
tests/test_linear_q8_gpu.py streams past the tokens instead)."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from dense_helpers import check
from gpu_helpers import DEV, Guarded, say
from linear_q8_sizes import TILES
from rows_helpers import linear_q8_64
from test_linear_q8_gpu import DT, gen, layer, normal, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


@pytest.mark.parametrize("T,k,n,tile,gated,split", TILES)
def test_every_tile_against_64_bits(T, k, n, tile, gated, split):
    for act, out, kind in (("silu" if gated else "gelu", "bf16", "i8"), ("relu" if gated else "none", "f32", "f16")):
        say(f"linear q8 T={T} k={k} n={n} tile {tile} gated={gated} split={split} {act} {kind} -> {out}")
        g = gen(T + k + n)
        lin = layer(g, n, k, gated, True, act)
        x, sx, q, s = tokens(g, T, k, kind)
        r = normal(g, (T, n), DT[out])
        y = Guarded((T, n), DT[out])
        nbytes = moe.workspace_size(moe.OP_LINEAR_Q8, T, k, n, moe._row_dt(x), 0, 0)
        assert nbytes > 0 or not split
        ws = Guarded((max(nbytes, 16),), torch.uint8)
        moe.linear_q8_forward(lin, x, x_scale=sx, residual=r, y=y.t, ws=ws.t)
        again = moe.linear_q8_forward(lin, x, x_scale=sx, residual=r, out_dtype=DT[out])
        torch.cuda.synchronize()
        y.check("y")
        ws.check("workspace")
        check(y.t, *linear_q8_64(q, s, lin, r, DT[out]), f"T={T} k={k} n={n}")
        assert torch.equal(y.t, again), "two runs differ"


# (T, k, n, gated) with n a multiple of 4, so that outputs may go by fours
QUADS = [(130, 400, 2152, True), (276, 448, 11212, False), (67, 2736, 1364, True), (68, 4816, 4224, False),
         (70, 15984, 4324, False), (2000, 1136, 2048, False)]


@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("T,k,n,gated", QUADS)
@pytest.mark.parametrize("left,stride,scale_at", [(64, 128, 0), (62, 128, 0), (61, 128, 0), (64, 129, 0), (64, 128, 1)])
def test_strides_and_in_place(T, k, n, gated, left, stride, scale_at, out):
    """y and residual in one column range of a wider matrix, the weights' scales at any address, aligned
    for reads of four or not; the columns beside it stay as they were."""
    g = gen(T + n + left)
    lin = layer(g, n, k, gated, True, "silu")
    lin.w_scale = torch.cat([lin.w_scale.new_zeros(scale_at), lin.w_scale])[scale_at:]
    x, s, _, _ = tokens(g, T, 3 * k, "i8")
    x = x[:, k:2 * k]
    wide = normal(g, (T, n + stride), DT[out])
    before = wide.clone()
    y = wide[:, left:left + n]
    moe.linear_q8_forward(lin, x, x_scale=s, residual=y, y=y)
    check(y, *linear_q8_64(x, s, lin, before[:, left:left + n], DT[out]), f"T={T} left={left}")
    assert torch.equal(wide[:, :left], before[:, :left]) and torch.equal(wide[:, left + n:], before[:, left + n:])
