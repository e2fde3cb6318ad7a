"""Sizes shared by the tests of the expert products and of the head's loss: those that run on the GPU
are the ones whose kernels tests/test_training_cpu.py looks up."""

# head: rows, dim, vocabulary.  For bfloat16 tiles of 128 x 128 for the logits, then of 256 x 256; for binary32 of
# 256 x 128, then of 128 x 128; k in whole 16 bytes and not, several stages of it, a last tile of 131 columns.
HEAD_TILES = [(900, 200, 4227), (900, 333, 4227), (1030, 200, 7299), (1030, 333, 7299)]
HEAD_TILES_CAPS = {"bf16": [0.0, 15.0, 40.0], "f32": [0.0, 15.0]}

# the gradients' products on the largest tiles too, cut along k and not
HEAD_LARGE = [(6000, 1537, 6100), (5000, 1536, 12003)]

# more rows than are looked through for a tile's targets at a time (8192, on narrow tiles 4096), on each shape of grad_w
HEAD_LONG = [(9300, 1536, 8195), (9500, 400, 16000), (9500, 300, 9000), (9500, 45, 15000)]

# head: one element a thread, streamed, tiles of 32 rows
HEAD_SIZES = [
    (1, 1, 1), (1, 8, 2), (2, 3, 5), (1, 64, 1000), (5, 40, 257), (64, 64, 256), (65, 129, 1023), (300, 96, 2500),
    (257, 200, 4097),
]

# experts, at most 16 rows each on average and many of them of one: counts, in, out
FEW_TO_ONE = [
    ([0] * 9 + [200] + [3, 0] * 11, 768, 256),           # streamed, many blocks of rows an expert
    ([0] * 20 + [900] + [1] * 43, 264, 520),
    ([300] + [0] * 7 + [2] * 24, 1544, 2041),
]
