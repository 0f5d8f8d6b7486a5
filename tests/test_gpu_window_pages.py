"""Windowed attention over tables whose pages wholly before every row's window have been given back:
their entries name no page, and what lies in them belongs to others.  No row sees a key there, so
the outputs are the oracle's, the same to the bit as with the pages in place, and the status is 0.
"""

import numpy as np
import pytest
import torch

from test_gpu_operators import BF, DEV, Batch, _dev, _say

pytestmark = pytest.mark.gpu


def _release(b, window):
    """Take the pages out of the tables that no row of their request sees, and spoil what they hold."""
    gone = 0
    for i, (n, c) in enumerate(zip(b.new, b.ctx)):
        first = max(0, c - n - window + 1)                    # first key that the request's first row sees
        pages = b.table[i, : first // b.page].copy()
        b.table[i, : len(pages)] = -1
        gone += len(pages)
        at = _dev(pages.astype(np.int64))
        for t in (b.cache.k, b.cache.v):
            t[at] = 0x7F if b.fp8 else float("nan")
        if b.fp8:
            b.cache.k_scales[at] = b.cache.v_scales[at] = float("nan")
    b.d_table = _dev(b.table)
    return gone


WINDOWS = [  # new, cached, heads, kv, d, page, fp8, window
    ([1] * 4, [200, 333, 700, 64], 8, 2, 128, 16, False, 64),             # narrow tiles, one part
    ([1] * 3, [1000, 777, 90], 8, 8, 64, 32, True, 37),
    ([1] * 64, list(range(1000, 1064)), 8, 1, 64, 16, False, 512),        # every place of the window in a tile
    ([1] * 64, list(range(1000, 1064)), 8, 1, 64, 16, True, 1),
    ([1] * 2, [5000, 9000], 8, 2, 128, 16, False, 3001),                  # split
    ([1] * 2, [5009, 9000], 8, 2, 64, 16, True, 1030),
    ([1] * 4, [3000, 9, 4000, 777], 50, 2, 64, 16, True, 1001),           # 32 rows a tile
    ([3, 6, 50, 1], [900, 1500, 2000, 70], 16, 2, 128, 16, False, 300),   # one tile, two tiles and a chunk
    ([3, 6, 50, 1], [900, 1500, 2000, 70], 16, 2, 128, 16, True, 45),
    ([200, 3], [300, 400], 4, 2, 128, 16, False, 33),                     # wide tiles, one part
    ([300], [709], 2, 1, 64, 16, False, 500),
    ([257], [1000], 6, 2, 64, 16, True, 211),
    ([130], [2000], 4, 4, 128, 32, True, 700),
    ([600], [5003], 8, 1, 128, 16, False, 4500),                          # split
    ([600], [5003], 8, 1, 64, 16, False, 1),
    ([100], [3000], 8, 8, 128, 16, True, 1500),
]


@pytest.mark.parametrize("case", WINDOWS)
def test_attention_window_over_released_pages(case):
    new, cached, heads, kv, d, page, fp8, window = case
    _say(f"window over released pages {len(new)} {case[2:]}")
    b = Batch(new, cached, heads, kv, d, page, fp8, seed=5, pad=2, wide=1)
    kept = b.run(window).clone()
    b.check(kept, window, "pages in place")
    assert _release(b, window) > 0
    got = b.run(window)
    b.check(got, window, "pages released")
    assert torch.equal(got, kept)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,cached", [([1, 1], [1000, 300]), ([80], [900])])
def test_attention_window_reports_a_missing_page_inside(fp8, new, cached):
    # a page that the first row of the request still sees is missing: reported, and read as zeros
    window, page = 100, 16
    b = Batch(new, cached, 8, 2, 128, page, fp8, seed=6)
    first = b.ctx[0] - new[0] - window + 1
    entry = first // page
    b.table[0, : entry + 1] = -1
    for x in (b.keys[0], b.values[0]):
        x[:, : (entry + 1) * page] = 0.0
    b.d_table = _dev(b.table)
    b.check(b.run(window), window, "missing page inside the window", status=8)
