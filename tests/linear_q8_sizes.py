"""Sizes of the linear layer on 8-bit integers that between them reach every tile kernel.

(T, k, n, tile, gated, split): the tile (tokens x weight rows) that the layer takes at
these sizes, and whether it splits k over workgroups.  k is never a multiple of 128 but in
the first of the last two, and fills at least four blocks of 128 a part."""

from linear_sizes import TILES as WIDE

TILES = [(T, 2 * k, n, tile, gated, split) for T, k, n, tile, gated, split in WIDE]
