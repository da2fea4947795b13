"""Sizes of 4-bit products of few rows by the kernel that the library chooses,
which tests/test_experts_launch_arguments.py pins on the CPU and whose results
tests/test_gpu_experts4_shapes.py checks: (blocks of 16 rows, waves along k,
waves) -> (rows, columns, the experts' offsets or None).  Rows and columns end
inside a tile."""


def experts(T, G):
    """Offsets of uneven groups, the third without a row; two rows of no group in
    front where there are more rows than groups."""
    front = 2 if T > G else 0
    bounds = [front + (T - 2 * front) * g // G for g in range(G + 1)]
    if G > 2:
        bounds[3] = bounds[2]
    return bounds


SHAPES = {
    (1, 8, 8): [(1, 4096, None), (16, 4087, None), (5, 40, None), (8, 500, experts(8, 64))],
    (1, 4, 8): [(7, 5003, None), (32, 2500, None), (8, 1024, experts(8, 64)), (90, 200, experts(90, 40))],
    (1, 2, 8): [(3, 9001, None), (31, 6007, None), (8, 2003, experts(8, 64))],
    (1, 1, 8): [(16, 17003, None), (17, 9001, None), (300, 1003, experts(300, 40))],
    (2, 4, 8): [(64, 1000, None), (33, 72, None), (125, 1003, None), (200, 500, experts(200, 8))],
    (2, 2, 8): [(128, 2301, None), (200, 1003, experts(200, 8))],
    (2, 1, 8): [(800, 500, experts(800, 32))],
    (3, 4, 8): [(33, 6007, None), (48, 8192, None)],
    (3, 4, 16): [(33, 11008, None), (48, 9001, None), (41, 8200, None)],
    (4, 4, 8): [(64, 6007, None), (127, 3001, None), (400, 600, experts(400, 8))],
    (4, 2, 8): [(49, 9001, None), (100, 5003, None), (400, 1003, experts(400, 8))],
    (4, 1, 8): [(64, 17003, None), (128, 9001, None), (400, 2003, experts(400, 8))],
}
# K of reads in whole aligned pieces (2), and wherever they begin (1).
READS = {2: [504, 2040, 2048], 1: [515, 2047]}
