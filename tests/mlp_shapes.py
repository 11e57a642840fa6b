"""Sizes of the feed-forward block for the tests of its tiles, (tokens, dim, hidden)."""

# fp32 sums of more products than a tile of 256 x 256 takes, at sizes that have tiles of 256 x 256
# for every CU: along the width (4096), the hidden width (2 x 8192) and the tokens
LONG_F32 = [(2048, 4096, 8192), (8192, 1024, 1024)]

# every tile of every product in both types, with and without split sums (test_mlp_tiles.py); widths
# that are whole chunks of 16 bytes and others, ragged in every direction
TILES = [(49, 36, 38), (2850, 36, 336), (193, 2195, 504), (2732, 2396, 54), (5727, 147, 2768),
         (12784, 2211, 94), (21, 1065, 5512), (983, 136, 4181), (4100, 1032, 2050), (8200, 256, 4100)]
