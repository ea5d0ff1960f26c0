"""Shapes that take a chosen path of the cache operators: the GPU tests run
them, and the host tests check that their plans take that path."""

# Window attention, bf16, on the tcgen05 kernel with two row tiles per CTA
# (key lists of more than 1792 keys):
# (b, hq, hkv, nq, nk, lens, window, sinks), whether the key list is split
TWO_TILES = [
    # causal only, an odd number of row tiles (the last CTA has no second one)
    ((1, 8, 2, 2500, 2500, [2500], 0, 0), False),
    # 7 heads a group (126 of 128 rows used), 130 first keys (a narrow second tile), a left-padded prompt
    ((2, 14, 2, 2100, 4300, [4300, 1500], 2000, 130), False),
    # one head a group: key tiles that only one of the two row tiles needs; an empty and a short sequence
    ((3, 4, 4, 300, 2900, [2900, 200, 0], 1900, 1), True),
    # 16 heads a group, 8 tokens a row tile, first keys that end inside a tile
    ((1, 16, 1, 257, 4000, [3990], 1800, 127), True),
    # short chunks on a long cache, in many pieces, without and with first keys
    ((2, 8, 2, 40, 6000, [6000, 5990], 0, 0), True),
    ((1, 8, 2, 40, 6000, [5990], 4000, 130), True),
    # a window that has just left the first keys behind; first keys that reach into it
    ((1, 32, 8, 1000, 2600, [2599], 1900, 700), False),
]

# Decode, bf16, with one full sequence among short ones, on the flat list of key
# tiles: (b, hq, hkv, nq, nk)
SKEWED = [(37, 32, 8, 1, 2500), (74, 28, 4, 3, 900), (33, 8, 1, 2, 12000)]

# Drafts of up to 16 tokens with more rows than one decode job holds, bf16:
# (b, hq, hkv, nq, nk, lens, window, sinks)
WIDE_DRAFTS = [
    (2, 28, 4, 16, 5000, [5000, 3], 0, 0),
    (3, 16, 1, 5, 700, [700, 0, 4], 100, 7),
    (2, 32, 2, 16, 2600, [2600, 1201], 1900, 130),
    (9, 28, 4, 10, 300, [300, 10, 9, 0, 1, 299, 150, 64, 65], 0, 0),
]

# fp32 calls whose CTAs take many key tiles each: (b, hq, hkv, nq, nk), key tiles of a CTA
LONG_RUNS_DECODE = ((37, 8, 8, 1, 131072), 4096)       # cache_decode_fp32.cu, 32 keys a tile
LONG_RUNS_TILE = ((150, 12, 1, 3, 131072), 2048)       # cache_tile.cu, 64 keys a tile
