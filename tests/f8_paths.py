"""Sizes of 8-bit floating point products that between them reach every kernel and every way of cutting
the work (which a CPU test checks against the library's own choice)."""

# (M, N, K): the product, plain, at 256 compute units
PRODUCTS = [
    (5, 500, 8208), (33, 500, 8192), (17, 1000, 8320), (32, 1100, 8208), (50, 700, 1040),       # few tokens, K in 4, 4, 2, 1, 1
    (64, 8200, 272),                                                                            # 64 tokens in tiles
    (74, 127, 416), (72, 8789, 144), (145, 11305, 144), (4388, 385, 160), (211, 11105, 144),     # the tile shapes
    (69, 1030, 8208), (128, 770, 4112), (222, 154, 4784), (1272, 183, 4112), (3000, 130, 2064),  # K in parts
    (1684, 6922, 272), (3000, 6150, 640),                                                       # large tiles
    (1553, 10293, 528), (1668, 9460, 544),                                                      # cut by tokens, by columns
]
# likewise, gated, with fp16 and with e4m3 output
GATED = [
    (3, 1030, 1040), (40, 700, 2064), (33, 8250, 272), (74, 127, 416), (272, 6042, 144), (145, 11305, 144), (72, 8789, 144),
    (69, 1030, 4112), (128, 770, 4112), (222, 154, 2064), (1272, 183, 4112),
    (211, 11105, 144), (466, 8250, 1040), (2058, 7698, 1040), (1261, 7091, 1088), (4403, 9491, 1040), (4805, 8624, 1072),
]
