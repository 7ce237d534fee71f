"""Shapes of the block-128 and grouped products with the kernel and tile that each is run by:
(CTAs a tile, rows of x a tile, K splits).  test_grouped_plan_cpu.py holds them to the library's choice."""

PAIR = (2, 256, 1)

# M, N, K: last tiles of 1, 3, 44 to 256 rows, N and K that end inside a block, more tiles than CTAs
DENSE = [
    ((515, 4104, 400), PAIR), ((256, 14336, 4096), PAIR), ((1030, 4104, 400), PAIR), ((129, 14344, 528), PAIR),
    ((385, 20488, 272), PAIR), ((2049, 1032, 272), PAIR), ((600, 4104, 16), PAIR),
    ((1000, 2056, 400), (1, 128, 1)), ((100, 20488, 272), (1, 128, 1)), ((65, 39944, 400), (1, 128, 1)),
    ((40, 20488, 272), (1, 64, 1)), ((33, 39944, 272), (1, 64, 1)), ((48, 14344, 1040), (1, 64, 1)),
    ((20, 20488, 272), (1, 32, 1)), ((32, 39944, 144), (1, 32, 1)),
    ((9, 20488, 272), (1, 16, 1)), ((16, 39944, 144), (1, 16, 1)),
]

# B, M, N, K
BATCHED = [((16, 512, 1024, 512), PAIR), ((16, 129, 2056, 272), PAIR), ((32, 300, 520, 272), PAIR),
           ((16, 257, 1032, 272), (1, 128, 1)), ((8, 257, 1032, 400), (1, 128, 1))]

# rows of each group around the edges of a pair's tile and of its CTAs' halves, groups without rows
EDGES = [1, 127, 0, 128, 129, 255, 256, 257, 513]
# rows of each group, N, K (a multiple of 128: both formats)
GROUPED = [((*EDGES, 0, *EDGES), 1032, 384, PAIR), ((*EDGES, 1500), 2056, 256, PAIR), ((700, 0, 0, 2000, 31, 3), 1032, 1152, PAIR),
           ((0, *EDGES), 4104, 128, PAIR), (tuple(EDGES), 520, 384, (1, 128, 1)), ((300, 0, 129, 200), 1032, 640, (1, 128, 1))]
# fp8_128 alone: a last block of 16 to 112 along K
GROUPED_RAGGED_K = [((*EDGES, 0, *EDGES), 1032, 400, PAIR), ((*EDGES, 1500), 2056, 144, PAIR), ((700, 0, 0, 2000, 31, 3), 1032, 1264, PAIR)]
