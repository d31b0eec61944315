"""Sizes at which lora_add's second half walks more than one block of rows or
columns, and takes more units of work than it has workgroups (256 compute
units).  (M, K, N, r, sizes of the adapters' groups; the other rows use none.)"""
from random import Random


def _few(seed, groups, most):
    rng = Random(seed)
    return [rng.randint(0, most) for _ in range(groups)]


# many rows of an adapter: rows a workgroup walks, whether a workgroup takes several units
ROWS = [
    (2000, 72, 2056, 64, [1100, 0, 770], 32, False),
    (900, 40, 2568, 128, [500, 333], 32, False),
    (2100, 264, 4104, 16, [700, 1300, 1], 48, False),
    (4100, 72, 7176, 16, [129, 900, 0, 1500, 257, 640, 33, 400], 128, True),
    (4100, 72, 7176, 64, [129, 900, 0, 1500, 257, 640, 33, 400], 128, True),
    (1200, 40, 11272, 96, [450, 390, 260], 128, True),
    (1200, 40, 11272, 128, [450, 390, 260], 128, True),
    (131200, 8, 8, 128, [70000, 61000], 128, True),      # more than 2^24 middle sums
]
# few rows of an adapter: column tiles a workgroup walks, whether it takes several units
COLUMNS = [
    (600, 72, 6288, 32, _few(1, 40, 28), 3, False),
    (600, 40, 6288, 64, _few(2, 40, 28), 4, False),
    (600, 40, 6288, 96, _few(3, 40, 28), 4, False),
    (600, 264, 6288, 128, _few(4, 40, 28), 7, False),
    (23000, 8, 264, 8, [17 + i % 5 for i in range(1023)], 2, True),
]
