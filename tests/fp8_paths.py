"""Sizes that reach each kernel of the FP8 block-scaled product, and the launch rule that says so
(gemm_fp8.hip and gemm_fp8_tiled.hip, written out again: a case that a changed rule sends elsewhere
fails in test_fp8_paths.py)."""
import numpy as np

from fp8_ref import blocks


def ceil(a, b):
    return -(-a // b)


def kernel(m, E, n, k, dtype):
    """The kernel that a call of m rows, E experts, n columns and k takes, by its template arguments."""
    exact = dtype == "fp32"
    most, rows = min(m, E), ceil(m, E)
    tiles = (m // 64 + most) * ceil(n, 128)
    if m < 4 * E or tiles < 96 or (rows <= 64 and tiles < 224):
        if rows > 16:
            return "stream 4 4" if rows > 64 else "stream 4 2" if rows > 32 else "stream 2 2"
        items = (m // 16 + most) * ceil(n, 16)
        assert items <= 1 << 21
        return "stream 1 1" if items <= 320 else "stream 2 1" if items <= 640 else "stream 4 1"
    avg = m // E
    low = avg < 96 or (m // 128 + most) * ceil(n, 128) < 512
    if not exact and blocks(k) <= 4:
        tiles = (m // (64 if low else 128) + most) * ceil(n, 128)
        if tiles >= 1024:
            return f"short {64 if low else 128} span {tiles // 512 if tiles < 2048 else 4}"
    if low:
        return "tile 64 exact" if exact else "tile 64 three stages" if blocks(k) >= 32 else "tile 64"
    big = ceil(m, 256) * ceil(n, 256)
    if not exact and avg >= 384 and big >= 224 and (big % 256 == 0 or big % 256 >= 160 or big >= 1024):
        return "tile 256"
    return "tile 128 exact" if exact else "tile 128"


# Experts of uneven rows, some without any; last tiles of one row, of a few and of nearly all.
UNEVEN = [1, 0, 130, 64, 257, 33, 0, 90, 65, 200, 12, 128]
TALL = [513, 0, 316, 386, 1024, 1, 770, 630]

# kernel -> (rows of the experts or None: dense rows, n, k, type).  K ends inside a block of 128
# and n inside a tile everywhere.
PATHS = {
    "stream 1 1": ([5, 0, 12, 3], 130, 272, "fp32"),
    "stream 2 1": ([5, 0, 12, 3] * 4, 300, 272, "bf16"),
    "stream 4 1": ([2, 0, 3, 1] * 20, 301, 272, "fp16"),
    "stream 2 2": ([30, 0, 41, 22], 301, 400, "fp32"),
    "stream 4 2": ([66, 0, 91, 33], 302, 400, "bf16"),
    "stream 4 4": ([101], 700, 144, "fp16"),
    "tile 64": (UNEVEN, 2301, 1040, "bf16"),
    "tile 64 three stages": (UNEVEN, 2300, 4240, "fp16"),
    "tile 64 exact": (UNEVEN, 2302, 656, "fp32"),
    "tile 128": ([1030, 129, 1, 0, 500], 4101, 784, "fp16"),
    "tile 128 exact": ([1030, 129, 1, 0, 500], 4100, 272, "fp32"),
    "tile 256": (TALL, 3843, 1040, "bf16"),
    "short 64 span 2": ([30, 0, 64, 12, 1, 65] * 5, 4001, 400, "bf16"),
    "short 64 span 3": ([30, 0, 64, 12, 1, 65] * 5, 5200, 240, "fp16"),
    "short 64 span 4": ([30, 0, 64, 12, 1, 65] * 5, 8100, 272, "bf16"),
    "short 128 span 2": (TALL, 5004, 112, "fp16"),
    "short 128 span 3": (TALL, 6130, 400, "bf16"),
    "short 128 span 4": ([900], 32770, 240, "bf16"),
}


def offsets(name):
    return np.concatenate(([0], np.cumsum(PATHS[name][0])))
