"""The windowed decode's block lookup: the block of a 16-token tile as the upper half of
a product, for every block size and up to the longest table."""
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _lookup(tile, n):
    magic = np.uint64((2 ** 32 + n - 1) // n)
    return (tile.astype(np.uint64) * magic) >> np.uint64(32)


def test_block_of_a_tile():
    with open(os.path.join(ROOT, "include", "pagedkv_window.h")) as f:
        tiles = int(re.search(r"PKV_WINDOW_MAX_TOKENS (0x[0-9a-f]+)", f.read()).group(1), 16) // 16
    with open(os.path.join(ROOT, "paged_kv_cache_212_gb300", "csrc", "window.h")) as f:
        most = int(re.search(r"kMaxBlockSize = (\d+);", f.read()).group(1)) // 16
    assert most == 16
    for n in range(2, most + 1):
        # what the product is above the quotient grows with the tile: the last million, and samples before
        at_end = np.arange(tiles - 2 ** 20, tiles + 1, dtype=np.int64)
        block = np.arange(0, tiles // n, 997, dtype=np.int64) * n          # the first tiles of blocks, and the last ones
        for tile in (at_end, block, block + n - 1):
            assert np.array_equal(_lookup(tile, n), (tile // n).astype(np.uint64)), n
    # the bound is the comment's: beyond 32 tiles a block the product goes wrong at this length
    tile = np.arange(tiles - 200, tiles + 1, dtype=np.int64)
    assert any((_lookup(tile, n) != (tile // n).astype(np.uint64)).any() for n in range(33, 200))
