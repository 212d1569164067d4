"""Sizes (M, K, N) of conv_linear by the form of the product that they reach.
test_channel_launches_cpu.py holds them to it; the GPU tests run them."""

# tiles of CTA pairs, finished in the kernel that sums them: 256 columns, 128,
# several to a pair, with odd edges
PAIR_TILES = [(19712, 64, 520), (20000, 96, 100), (39001, 72, 136), (5000, 512, 1030)]
# single CTAs with tiles of more than 64 columns
WIDE_SINGLE_TILES = [(10240, 64, 72), (10240, 64, 100), (16384, 128, 150), (16384, 128, 190), (10240, 72, 256)]
# fewer pair tiles than pairs, and sums long enough to cut: all in runs, joined
JOINED_RUNS = [(300, 20488, 520), (513, 30008, 130), (1000, 8200, 1000)]
# a short last round of pair tiles cut into runs
CUT_LAST_ROUND = [(5100, 2968, 1000), (4990, 4104, 1250)]
# one tile's sum shared by the CTAs of a cluster
CLUSTERS = [(8, (128, 4096, 128)), (8, (200, 2048, 100)), (4, (700, 1024, 256)), (2, (1100, 520, 500)),
            (8, (64, 8200, 500)), (2, (16, 1032, 9000))]
# up to four rows, on the CUDA cores
FEW_ROWS = [(1, 8195, 67), (2, 1003, 300), (3, 4096, 129), (4, 2055, 1000)]
