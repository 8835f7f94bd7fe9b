"""Sizes of the feed-forward products that reach kernels which the other sizes in the tests leave out: K divided, 64 x 128
tiles by expert, 32 rows and columns of the kernel for few rows, blocks of several experts in parts.

Each entry: sizes, then for a 16-bit and for a float32 C the kernel that they are to reach, as tests/test_feed_forward_paths.py
checks against the rule itself.
"""

# (M, N, K)
LINEAR = [((100, 500, 4096), "tile 64x64 divided", "tile 64x64 divided"),
          ((64, 513, 7168), "tile 64x64 divided", "tile 64x64 divided"),
          ((40, 301, 4096), "tile 64x64 divided", "tile 64x64 divided"),
          ((18, 4123, 7040), "tile 64x128 divided", "rows 32x16"),
          ((33, 5953, 4992), "tile 64x64", "tile 64x128 divided"),
          ((456, 2075, 5792), "tile 64x128", "tile 128x128 divided"),
          ((32, 7168, 2048), "rows 32x32", "rows 32x32"),
          ((17, 6300, 400), "rows 32x32", "rows 32x32")]

# (sizes of the groups, N, K, rows before and behind them)
GROUPED = [(([300, 0, 690], 1024, 512, 0, 10), "tile 64x128", "tile 64x128"),
           (([20, 0, 9, 12, 0, 31, 3, 7, 0, 0, 20] * 3, 114, 400, 3, 28), "rows 32x32", "rows 32x32"),
           (([30, 0, 33], 2000, 272, 0, 1), "rows 32x32", "rows 32x32"),
           (([2, 3, 0, 4, 1, 0, 1] * 5, 463, 144, 12, 11), "tile 64x128", "tile 64x128")]

# (sizes of the groups, M, N, rows before and behind them); float32 C
DEEP = [(([6000, 0, 9000], 70, 130, 0, 0), "tile 64x64 divided"),
        (([4000, 0, 4100, 1], 64, 64, 0, 0), "tile 64x64 divided"),
        (([9000, 0, 9000, 1], 200, 101, 3, 0), "tile 64x64 divided"),
        (([8000, 0, 1, 8000, 500], 10, 804, 0, 16), "tile 64x128 divided"),
        (([14000, 0, 15000, 100, 80], 73, 1628, 0, 0), "tile 128x128 divided")]


def blocks(sizes, head, tail):
    """Blocks of 128 rows that the groups can have at most."""
    T = sum(sizes) + head + tail
    return (T + 127 * min(T, len(sizes))) // 128
