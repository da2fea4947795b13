"""Sizes of grouped products whose kernels tests/test_experts_launch.py pins on
the CPU and whose results tests/test_gpu_experts_tiles.py checks: (T, K, N,
offsets) by the side of the tile that the library chooses."""

# Full tiles, tiles of few rows, the last tiles of a grid in halves, groups of
# no rows, odd and even counts of slices, the last one whole and ragged.
PRODUCTS = {
    256: [(2000, 1032, 6152, [0, 100, 1990]), (4100, 1032, 4104, [3, 1300, 4100]), (2100, 1088, 8200, [0, 0, 2100]),
          (1300, 2056, 8200, [0, 129, 1300])],
    128: [(520, 136, 2056, [0, 129, 130, 385, 520]), (333, 520, 2056, [0, 100, 101, 101, 329]), (520, 264, 4104, [0, 17, 145, 145, 520]),
          (1000, 128, 4104, [0, 500, 628, 756, 1000])],
    16: [(8, 2048, 1024, [0, 1, 1, 2, 5, 8]), (20, 264, 72, [0, 17, 17, 20]), (1, 8, 8, [0, 1]), (40, 4096, 200, [0, 3, 20, 39]),
         (70, 136, 40, list(range(0, 71))), (300, 136, 264, [0, 99, 100, 300])],
}
GRADIENTS = {
    256: [(2000, 1544, 4104, [0, 1, 2000]), (3000, 1032, 4104, [5, 1029, 1029, 2990]), (1500, 4104, 4104, [0, 1499])],
    128: [(1000, 1544, 1288, [0, 3, 500, 500, 990]), (333, 520, 264, [0, 100, 101, 101, 229, 333]), (70, 96, 40, [3, 10, 10, 61, 66])],
}
