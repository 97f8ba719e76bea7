"""The 8-bit linear layer's streams of wide layers against 64 bits: four groups of rows a wave (17 to 32 tokens)
and two slices of k a workgroup, which narrow layers do not take."""
import pytest
import torch

import activation_sparse_expert_amd as moe
from dense_helpers import check
from gpu_helpers import Guarded, say
from rows_helpers import linear_q8_64
from test_linear_q8_gpu import DT, gen, layer, normal, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


# Two slices where 16 outputs a wave and two slices give 1536 waves: from 12273 outputs, 14401 here.  Four
# groups a wave where 64 outputs (gated 32) and two slices give 896: from 28672 outputs (gated 14336), 28705
# and 14401 here, and the numbers just below.  k: one block and a part, many blocks, fewer blocks than slices,
# more than the ring holds; multiples of 128 and not.
@pytest.mark.parametrize("k", [16, 112, 272, 1040, 2048])
@pytest.mark.parametrize("T,n,gated", [
    (1, 14401, False), (1, 14401, True), (2, 14401, False), (2, 14401, True), (8, 14401, False), (8, 14401, True),
    (9, 14401, False), (16, 14401, True), (16, 14401, False), (1, 12272, False), (1, 12288, True),
    (17, 14401, True), (24, 14401, True), (25, 14401, True), (32, 14401, True), (32, 14335, True), (24, 14336, True),
    (17, 28705, False), (24, 28705, False), (25, 28705, False), (32, 28705, False), (24, 28672, False), (32, 28671, False)])
def test_wide_layers(T, n, gated, k):
    for i, (kind, bias, res, act, out) in enumerate([("i8", False, False, "none", "f32"), ("bf16", True, True, "silu", "bf16"),
                                                     ("f32", False, True, "relu", "f32"), ("f16", True, False, "gelu", "f16")]):
        if T > 1 and i > 1:
            break                                       # (tokens of 16 and 32 bits go the same way then)
        say(f"linear q8 stream T={T} k={k} n={n} {kind} gated={gated}")
        g = gen(100 * i + T + k + n)
        lin = layer(g, n, k, gated, bias, act)
        x, sx, q, s = tokens(g, T, k, kind)
        r = normal(g, (T, n), DT[out]) if res else None
        y = Guarded((T, n), DT[out])
        ws = Guarded((moe.workspace_size(moe.OP_LINEAR_Q8, T, k, n, moe._row_dt(x), 0, 0),), torch.uint8)
        assert moe.linear_q8_plan(T, k, n, gated) == (None, 0), "streamed"
        moe.linear_q8_forward(lin, x, x_scale=sx, residual=r, y=y.t, ws=ws.t)
        torch.cuda.synchronize()
        y.check("y")
        ws.check("workspace")
        check(y.t, *linear_q8_64(q, s, lin, r, DT[out]), f"T={T} k={k} n={n} {kind} gated={gated}")
        if kind != "i8":
            given = moe.linear_q8_forward(lin, q, x_scale=s, residual=r, out_dtype=DT[out])
            assert torch.equal(y.t, given), "codes made in the call and given"


# 13056 fp32 and 21504 16-bit numbers are the longest token whose numbers and codes have room beside the weights'
# (64 KiB of LDS); the next ones have a launch of their own.  40 outputs go by eight slices of such k, whose
# rings then fill the rest of LDS; 14336 + 14336 by two.
@pytest.mark.parametrize("n,gated", [(14336, True), (40, True), (40, False), (9000, True)])
@pytest.mark.parametrize("k,kind", [(128, "bf16"), (4112, "bf16"), (8192, "f16"), (8192, "f32"), (13056, "f32"), (13072, "f32"),
                                    (21504, "bf16"), (21504, "f16"), (21520, "bf16")])
def test_one_token_whose_codes_the_product_makes(k, kind, n, gated):
    g = gen(k + n)
    lin = layer(g, n, k, gated, True, "silu")
    x, _, q, s = tokens(g, 1, k, kind)
    y = moe.linear_q8_forward(lin, x, out_dtype=DT["bf16"])
    check(y, *linear_q8_64(q, s, lin, None, DT["bf16"]), f"k={k} {kind}")
    assert torch.equal(y, moe.linear_q8_forward(lin, q, x_scale=s, out_dtype=DT["bf16"]))
