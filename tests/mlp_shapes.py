"""Sizes of the feed-forward block for the tests of its tiles, (tokens, dim, hidden)."""

# fp32 sums of more products than a tile of 256 x 256 takes, at sizes that have tiles of 256 x 256
# for every CU: along the width (4096), the hidden width (2 x 8192) and the tokens
LONG_F32 = [(2048, 4096, 8192), (8192, 1024, 1024)]
