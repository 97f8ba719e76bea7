"""Sizes of the linear layer on 8-bit integers that between them reach every tile kernel.

(T, k, n, tile, gated, split): the tile (tokens x weight rows) that the layer takes at
these sizes, and whether it splits k over workgroups.  k is a multiple of 128 in the last two
only."""

TILES = [
    (77, 400, 4153, (64, 64), False, False), (130, 400, 2153, (64, 64), True, False),
    (34, 17120, 3, (64, 64), False, True), (70, 17120, 9, (64, 64), True, True),
    (34, 352, 17683, (64, 128), False, False), (38, 336, 8565, (64, 128), True, False),
    (33, 5264, 2475, (64, 128), False, True), (77, 2736, 1363, (64, 128), True, True),
    (17165, 1008, 73, (128, 128), False, False), (18331, 1136, 35, (128, 128), True, False),
    (73, 12848, 2525, (128, 128), False, True), (2759, 12992, 33, (128, 128), True, True),
    (12185, 304, 265, (128, 256), False, False), (17812, 320, 107, (128, 256), True, False),
    (70, 15984, 4323, (128, 256), False, True), (73, 12848, 2525, (128, 256), True, True),
    (44819, 368, 129, (256, 256), False, False), (1100, 368, 11213, (256, 256), False, False),
    (1500, 304, 12077, (256, 256), True, False),
    (300, 4096, 4096, (64, 128), False, False), (300, 14336, 4096, (128, 256), False, True),
]
