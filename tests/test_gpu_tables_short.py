"""Block tables when the free pages run out: a request whose pages are not there takes none, and the
requests behind it are served from what the served ones ahead of them left."""

import numpy as np
import pytest
import torch

import dequant_gemv_w4_amd as w4
import oracle
from test_gpu_operators import DEV, _dev, _say

pytestmark = pytest.mark.gpu


def _check(new, lens, free, count, table, page, tokens, in_place):
    new, lens, free, table = (np.ascontiguousarray(x, dtype=np.int32) for x in (new, lens, free, table))
    cu, pos, slots, lens_ref, left, table_ref, status = oracle.block_tables_ref(new, lens, free, count, table, page, tokens)
    d_lens, d_count, d_table = _dev(lens), _dev(np.array([count], np.int32)), _dev(table)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = {} if in_place else dict(lens_out=torch.full_like(d_lens, -9), free_count_out=torch.full_like(d_count, -9))
    got = w4.w4_block_tables(_dev(new), d_lens, _dev(free), d_count, d_table, page, tokens=tokens, status=st, **kw)
    assert got[0].cpu().tolist() == cu
    assert kw.get("lens_out", d_lens).cpu().tolist() == lens_ref
    assert int(kw.get("free_count_out", d_count)) == left
    assert got[1].cpu().tolist() == pos
    assert got[2].cpu().tolist() == slots
    assert d_table.cpu().tolist() == table_ref
    assert int(st) == status
    return lens_ref, left, status


@pytest.mark.parametrize("in_place", [False, True])
def test_requests_behind_one_that_is_short(in_place):
    # five pages: ten are not there, one and one are
    got = _check([160, 1, 16], [0, 0, 0], range(5), 5, np.full((3, 12), -1), 16, 200, in_place)
    assert got == ([0, 1, 16], 3, 32)
    # the first that does not fit is not the last: 3 of 4 go, 2 do not, 1 goes, 1 does not, none are asked, 0 are left
    got = _check([48, 32, 7, 16, 5], [0, 0, 16, 0, 3], [9, 8, 7, 6], 4, np.array([[-1] * 4, [-1] * 4, [1, -1, -1, -1], [-1] * 4, [2, -1, -1, -1]]),
                 16, 120, in_place)
    assert got == ([48, 0, 23, 0, 8], 0, 32)


@pytest.mark.parametrize("B,most,share,tokens_more", [(3, 300, 0.3, 0), (64, 200, 0.5, 5), (65, 200, 0.5, 0), (300, 60, 0.7, 3), (1025, 90, 0.6, 0),
                                                      (4096, 40, 0.4, 9), (4096, 40, 0.0, 0), (500, 100, 0.5, -900)])
@pytest.mark.parametrize("in_place", [False, True])
def test_short_of_pages(B, most, share, tokens_more, in_place):
    _say(f"tables short of pages {B} {most} {share} {tokens_more}")
    rng = np.random.default_rng(B + most)
    page = 16
    # a few large requests between many small ones
    new = np.where(rng.random(B) < 0.1, rng.integers(0, 8 * most + 1, B), rng.integers(0, most // 8 + 1, B))
    lens = rng.integers(0, 100, B)
    new[0], lens[1] = most, 16
    if B > 60:
        new[20], lens[30] = -3, -1                            # not served for their lengths, whatever is free
    have, want = -(-np.maximum(lens, 0) // page), -(-(np.maximum(lens, 0) + np.maximum(new, 0)) // page)
    wide = max(1, int(want.max()) - (1 if B == 300 else 0))   # there also a table that is too narrow
    table = np.full((B, wide), -1)
    pool = rng.permutation(int(want.sum()) + 5)
    used = 0
    for b in range(B):
        table[b, : have[b]] = pool[used: used + have[b]]
        used += have[b]
    count = int(share * (want - have).sum())
    tokens = max(1, int(np.maximum(new, 0).sum()) + tokens_more)
    lens_ref, left, status = _check(new, lens, pool[used:], count, table, page, tokens, in_place)
    assert status & 32 and left <= count
