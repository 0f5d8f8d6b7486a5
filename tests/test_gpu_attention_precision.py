"""Attention held more closely than a tolerance by size can: weights in two bfloat16 parts where few rows
are, and every key once, at the lengths and numbers of rows where tiles and parts change.

* Two kinds of keys, values +1 and -1, whose weights nearly cancel, and scores that one product and no
  sum makes: what the output is off by is what the weights are off by.  In two parts each is within 2^-16
  of itself, its score's rounding, exp2's argument and result within 8 u, sums of n terms in binary32 within
  n / 8 u on either side, u = 2^-24; the output is rounded by 2^-8 of itself, and itself is small.  A weight
  rounded to bfloat16 alone (these are 0.38 of 2^-8 off) is out by several times that.
* Scores of zero: all weights are 1 without rounding and the output is a share of keys.  A column counts
  every 64th or 128th run of 32 keys, so that a run left out or taken twice changes some column by a third
  at least, at any length tested here.  Beside the output's 2^-8 only the parts are rounded: a quotient and a
  product each, their sum (64 terms at most), a quotient and a product: 70 u, 80 u allowed.
"""

import numpy as np
import pytest
import torch

import oracle
from _util import to_np32
from test_gpu_operators import BF, DEV, U32, UB, Batch, _close, _dev, _say

pytestmark = pytest.mark.gpu


def _at(b, i):
    """Pages and places of a request's keys, on the device."""
    j = np.arange(b.ctx[i])
    return torch.from_numpy(b.table[i, j // b.page].astype(np.int64)).to(DEV), torch.from_numpy(j % b.page).to(DEV)


def _put(b, i, which, x):
    """x [ctx, kv, d], exact in E4M3, into a request's rows (with scales of 1)."""
    pg, at = _at(b, i)
    t = getattr(b.cache, which)
    if b.fp8:
        t[pg, :, at] = _dev(oracle.e4m3_encode(x))
        getattr(b.cache, which + "_scales")[pg, :, at] = 1.0
    else:
        t[pg, :, at] = _dev(x.astype(np.float32), BF)
    (b.keys if which == "k" else b.values)[i] = x.transpose(1, 0, 2)


NARROW = [  # new, cached, heads, kv, d, page, fp8, pad: requests of few rows
    ([1] * 3, [0, 40, 5000], 8, 1, 128, 16, False, 0),        # 16 rows a tile, one token a request
    ([1] * 3, [2, 700, 20000], 8, 2, 64, 16, True, 0),
    ([1] * 3, [40, 3000, 1200], 24, 1, 128, 16, False, 0),    # 32 rows a tile
    ([1] * 2, [6000, 900], 33, 1, 64, 16, True, 0),
    ([3], [700], 8, 1, 128, 16, False, 1),                    # few rows in all
    ([3, 60, 4, 1], [5000, 30, 900, 2500], 16, 2, 128, 16, False, 2),   # beside a chunk, 24, 32 and 8 rows
    ([6, 60, 5, 1], [5000, 30, 900, 2500], 16, 2, 128, 16, False, 2),   # 48 and 40 rows: two tiles
    ([6, 60, 5, 1], [5000, 30, 900, 2500], 7, 1, 64, 16, True, 2),
]


@pytest.mark.parametrize("case", NARROW)
def test_attention_weights_of_few_rows(case):
    new, cached, heads, kv, d, page, fp8, pad = case
    _say(f"weights of few rows {case}")
    b = Batch(new, cached, heads, kv, d, page, fp8, seed=17, pad=pad)
    b.scale, t = 1.0, -0.6875                                 # exp(t) = 0.50283: between two bfloat16 numbers
    b.q[:] = 0.0
    b.q[..., 0] = 1.0
    b.d_q = _dev(b.q, BF)
    for i, c in enumerate(b.ctx):
        k, v = np.zeros((c, kv, d)), np.ones((c, kv, d))
        low = np.arange(c) % 3 > 0
        k[low, :, 0], v[low] = t, -1.0
        _put(b, i, "k", k)
        _put(b, i, "v", v)
    got = to_np32(b.run())
    rounded = float(torch.tensor(np.exp(t)).to(BF))           # what one bfloat16 part would make of exp(t)
    assert abs(rounded / np.exp(t) - 1) > 0.35 * UB
    for i, n in enumerate(new):
        if n * heads // kv > 64:
            continue                                          # the chunk
        rows = slice(int(b.cu[i]), int(b.cu[i]) + n)
        ref, weight = oracle.attention_ref(b.q[rows], b.keys[i], b.values[i], b.ctx[i], b.scale)
        off = (2.0 ** -16 + 2 * (8 + b.ctx[i] / 8) * U32) * weight
        _close(got[rows], ref, off + UB * (np.abs(ref) + off), f"request {i}")


COUNTS = [  # new, cached, heads, kv, d, page, fp8, window
    ([300], [4500], 32, 8, 64, 64, False, 0),                 # a chunk past 4096 keys: more parts than below
    ([260, 1], [9000, 30], 8, 8, 128, 16, False, 0),
    ([120], [4200], 16, 2, 64, 16, True, 0),
    ([3, 6, 40], [3000, 2500, 9], 16, 2, 64, 16, False, 0),   # 24 rows, two tiles and a chunk
    ([3, 6, 40], [8000, 2500, 9], 16, 2, 128, 16, True, 0),
    ([1] * 3, [40, 3000, 1200], 24, 1, 128, 16, False, 0),    # 32 rows a tile
    ([1] * 2, [9000, 513], 40, 1, 64, 32, True, 0),
    ([1] * 3, [20000, 256, 511], 8, 1, 64, 64, False, 0),
    ([1] * 2, [5000, 9000], 8, 2, 64, 16, False, 3001),
    ([200, 3], [5000, 700], 4, 2, 64, 16, True, 500),
    ([300], [6000], 8, 1, 64, 16, False, 4999),
    ([4, 7, 50], [3000, 2500, 900], 8, 1, 128, 16, False, 700),
    ([2, 0, 1, 0], [3000, 5, 5000, 9], 8, 1, 64, 16, False, 0),   # fewer tokens than requests
    ([6, 0, 0, 0, 0, 0], [4100, 5, 6, 7, 8, 9], 8, 1, 64, 16, False, 0),   # as many, not one each
]


@pytest.mark.parametrize("case", COUNTS)
def test_attention_counts_runs_of_keys_once(case):
    new, cached, heads, kv, d, page, fp8, window = case
    _say(f"counts {case}")
    b = Batch(new, cached, heads, kv, d, page, fp8, seed=19)
    b.d_q.zero_()
    for i, c in enumerate(b.ctx):
        j = np.arange(c)
        v = np.zeros((c, kv, d))
        v[j, :, j // 32 % d] = 1.0
        _put(b, i, "v", v)
    got = to_np32(b.run(window))
    assert b.status == 0
    for i, n in enumerate(new):
        for t in range(n):
            last = b.ctx[i] - n + t
            first = max(0, last - window + 1) if window else 0
            ref = np.bincount(np.arange(first, last + 1) // 32 % d, minlength=d) / (last + 1 - first)
            row = got[int(b.cu[i]) + t]
            assert np.all(np.abs(row - ref) <= (UB + 80 * U32) * ref), (i, t)
