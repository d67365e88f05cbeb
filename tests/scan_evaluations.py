"""Sizes of the per-channel scan and the evaluation that each takes (not a test
module). tests/test_scan_plan.py holds the library's choice to this list, so that
the GPU tests that run it keep reaching what it says.

(batch, seq_len, dim, dstate, ngroups, with context_lengths): evaluation, which is
("rows", lanes of a channel), ("sweep", waves, sixteens of dstate) or
("chunks", sixteens, tokens of a chunk, chunks, chunks of a workgroup).
"""
SIZES = {
    # rows: up to four tokens, more, blocks cut short
    (16, 5, 1100, 16, 1, True): ("rows", 4),
    (64, 17, 600, 16, 1, True): ("rows", 4),
    (64, 20, 640, 16, 1, False): ("rows", 4),
    (2, 4, 70, 24, 1, True): ("rows", 8),
    (1, 5, 600, 20, 1, False): ("rows", 8),
    (1, 4, 1500, 32, 1, False): ("rows", 8),
    (2, 5, 60, 40, 1, True): ("rows", 16),
    (4, 5, 60, 64, 2, False): ("rows", 16),
    (2, 6, 33, 100, 1, True): ("rows", 32),
    (2, 4, 33, 128, 1, False): ("rows", 32),
    (1, 7, 20, 200, 1, True): ("rows", 64),
    (2, 3, 20, 256, 1, False): ("rows", 64),
    # sweeps of 4, 8 and 16 waves
    (64, 3, 40, 8, 1, True): ("sweep", 4, 1),
    (4, 60, 100, 16, 1, False): ("sweep", 4, 1),
    (8, 40, 1000, 24, 1, True): ("sweep", 4, 2),
    (5, 30, 60, 40, 1, True): ("sweep", 4, 3),
    (2, 31, 1864, 256, 1, True): ("sweep", 4, 16),
    (3, 100, 90, 16, 1, True): ("sweep", 8, 1),
    (2, 70, 130, 20, 2, True): ("sweep", 8, 2),
    (2, 75, 30, 40, 1, False): ("sweep", 8, 3),
    (2, 90, 30, 100, 1, True): ("sweep", 8, 7),
    (3, 123, 1051, 256, 1, False): ("sweep", 8, 16),
    (1, 2048, 5120, 16, 1, True): ("sweep", 8, 1),
    (1, 180, 100, 16, 1, True): ("sweep", 16, 1),
    (1, 170, 70, 24, 1, True): ("sweep", 16, 2),
    (1, 150, 70, 40, 1, False): ("sweep", 16, 3),
    (1, 170, 885, 128, 1, True): ("sweep", 16, 8),
    (1, 207, 2962, 256, 1, True): ("sweep", 16, 16),
    # chunks of 32 tokens, longer ones, two to a row, one to a row
    (1, 1100, 60, 16, 3, False): ("chunks", 1, 32, 35, 4),
    (1, 2048, 5120, 16, 1, False): ("chunks", 1, 56, 37, 4),
    (2, 3036, 2976, 4, 1, True): ("chunks", 1, 36, 85, 4),
    (2, 3036, 2976, 4, 1, False): ("chunks", 1, 96, 32, 4),
    (3, 194, 27325, 16, 1, False): ("chunks", 1, 100, 2, 2),
    (43, 21, 3568, 12, 1, False): ("chunks", 1, 21, 1, 1),
    (29, 34, 3390, 12, 1, False): ("chunks", 1, 34, 1, 1),
    (1, 1000, 256, 24, 1, False): ("chunks", 2, 32, 32, 4),
    (1, 1000, 256, 24, 1, True): ("chunks", 2, 32, 32, 4),
    (1, 4183, 2098, 20, 1, True): ("chunks", 2, 36, 117, 4),
    (14, 22, 4970, 20, 1, False): ("chunks", 2, 22, 1, 1),
    (1, 600, 256, 40, 1, False): ("chunks", 3, 32, 19, 4),
    (1, 600, 90, 40, 3, True): ("chunks", 3, 32, 19, 4),
    (1, 1348, 1560, 48, 1, False): ("chunks", 3, 36, 38, 4),
    (9, 18, 3940, 40, 1, False): ("chunks", 3, 18, 1, 1),
    (1, 986, 1617, 64, 1, False): ("chunks", 4, 36, 28, 4),
    (1, 300, 50, 80, 1, True): ("chunks", 5, 32, 10, 2),
    (1, 940, 904, 100, 1, False): ("chunks", 7, 36, 27, 2),
    (1, 557, 1430, 128, 1, False): ("chunks", 8, 36, 16, 2),
    (1, 140, 30, 200, 1, True): ("chunks", 13, 32, 5, 1),
    (4, 33, 1877, 200, 1, False): ("chunks", 13, 33, 1, 1),
    (2, 336, 526, 256, 1, False): ("chunks", 16, 36, 10, 1),
}

# One small size of each kind of kernel, for the pairs of types.
TYPED = {
    (16, 5, 1100, 16, 1, True): ("rows", 4),
    (1, 5, 600, 20, 1, False): ("rows", 8),
    (2, 6, 33, 100, 1, True): ("rows", 32),
    (4, 60, 100, 16, 1, False): ("sweep", 4, 1),
    (2, 75, 30, 40, 1, False): ("sweep", 8, 3),
    (1, 180, 100, 16, 1, True): ("sweep", 16, 1),
    (1, 1100, 20, 16, 1, False): ("chunks", 1, 32, 35, 4),
    (1, 300, 20, 64, 1, False): ("chunks", 4, 32, 10, 4),
    (1, 140, 30, 200, 1, True): ("chunks", 13, 32, 5, 1),
}
