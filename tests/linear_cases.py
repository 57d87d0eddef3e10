"""Sizes of the linear layer's products by the tiles that they are cut into.

(tokens, columns of the result, length of the sum) of products in tiles of 256,
and which tiles: whole ones, one block each, or split over several blocks.
"""
LARGE_TILES = {
    (3000, 4160, 1032): ("whole",), (3001, 4163, 1030): ("whole",),
    (1015, 4280, 6000): ("split",), (1271, 3251, 5999): ("split",),
    (4343, 4792, 6000): ("whole", "split"), (4599, 4531, 6001): ("whole", "split"),
}
