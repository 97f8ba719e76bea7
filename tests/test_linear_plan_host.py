"""Which kernels the linear layer's tests reach, without a GPU."""
import random

import pytest

import activation_sparse_expert_amd as moe
from linear_sizes import TILES
from test_api_host import _lib_or_skip


@pytest.mark.parametrize("T,k,n,tile,gated,split", TILES)
def test_sizes_reach_the_tile_they_name(T, k, n, tile, gated, split):
    _lib_or_skip()
    got, parts = moe.linear_plan(T, k, n, gated)
    assert got == tile and (parts > 1) == split
    assert not split or moe.workspace_size(moe.OP_LINEAR, T, k, n) > 0


def test_sizes_reach_every_tile_that_calls_can_take():
    """4000 sizes over the range: each (tile, gated, split or not) that any of them takes
    is one of the tested ones."""
    _lib_or_skip()
    tested = {(tile, gated, split) for _, _, _, tile, gated, split in TILES}
    rng = random.Random(7)
    for _ in range(4000):
        T, k, n = round(2 ** rng.uniform(5, 16)), 8 * round(2 ** rng.uniform(0, 14)), round(2 ** rng.uniform(0, 17))
        for gated in (False, True):
            tile, parts = moe.linear_plan(T, k, n, gated)
            assert tile is None or (tile, gated, parts > 1) in tested, (T, k, n, gated, tile, parts)


def test_few_tokens_stream_and_bad_sizes_are_refused():
    L = _lib_or_skip()
    assert moe.linear_plan(32, 4096, 14336) == (None, 0)
    assert moe.linear_plan(33, 8, 1) == (None, 0)
    assert L.moe_linear_plan(33, 4096, 14336, 0, None, None) > 0
    for T, k, n in ((0, 64, 64), (65537, 64, 64), (4, 60, 64), (4, 64, 0)):
        with pytest.raises(ValueError):
            moe.linear_plan(T, k, n)
