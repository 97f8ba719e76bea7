"""Sizes of the linear layer that between them reach every tile kernel.

(T, k, n, tile, gated, split): the tile (tokens x weight rows) that the layer
takes at these sizes, and whether it splits k over workgroups.  k is never a
multiple of 64 but in the first of the last two (a short prompt through a square
projection), and fills at least four blocks of 64 a part."""

TILES = [
    (36, 200, 2153, (64, 64), False, False), (36, 200, 2153, (64, 64), True, False),
    (38, 8344, 9, (64, 64), False, True), (38, 8344, 9, (64, 64), True, True),
    (66, 224, 9001, (128, 64), False, False), (70, 216, 4358, (128, 64), True, False),
    (2124, 8312, 10, (128, 64), False, True), (67, 1368, 1362, (128, 64), True, True),
    (725, 200, 10809, (128, 128), False, False), (2724, 200, 1409, (128, 128), True, False),
    (2587, 12312, 257, (128, 128), False, True), (2461, 11696, 138, (128, 128), True, True),
    (276, 224, 11211, (128, 256), False, False), (131, 200, 8387, (128, 256), True, False),
    (68, 2408, 4226, (128, 256), False, True), (33, 2072, 4263, (128, 256), True, True),
    (1439, 200, 5502, (256, 256), False, False), (276, 224, 11211, (256, 256), True, False),
    (300, 4096, 4096, (128, 256), False, True), (300, 4104, 4099, (128, 256), False, True),
]
