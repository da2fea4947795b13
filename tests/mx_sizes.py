"""Sizes whose launches tests/test_mx_launch.py pins on the CPU and whose
results tests/test_gpu_mx_tiles.py checks on the GPU."""
# (m, n, k) of products on 256 x 256 tiles: nine passes and one over four
# slices and the remainders after them, an odd last block, odd columns.
LARGE_PRODUCTS = [(3500, 3501, 2305), (3450, 3496, 1056)]
# (t, f, n) of gradients on 256 x 256 tiles, and the chunks of tokens that a
# bfloat16 or another dY is taken in (0: on smaller tiles).
LARGE_GRADS = {(333, 3500, 3496): (1, 1), (200, 3400, 3401): (1, 1), (2500, 1500, 1500): (0, 7)}
