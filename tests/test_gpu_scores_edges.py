"""GPU parity of attention with capped or biased scores at the ends of what its steps of keys may hold, against the
binary64 oracle (tolerances: _batch.Batch.check, where no other stands at the test).
"""

import numpy as np
import pytest

import dequant_gemv_w4_amd as w4
import oracle
from _batch import BF, Batch, dev

pytestmark = pytest.mark.gpu


def _scores(cap=0.0, slopes=None, first=None, prefix=None):
    return w4.W4Scores(cap=cap, slopes=None if slopes is None else dev(slopes), first_keys=None if first is None else dev(first),
                       prefix_lens=None if prefix is None else dev(prefix))


def _set_keys(b, i, j, codes):
    """Keys j of request i get the elements codes [len(j)] (of a bfloat16 cache; codes under the scales that an 8-bit one
    has), in the cache alone."""
    pg = dev(b.table[i, j // b.page].astype(np.int64))
    b.cache.k[pg, :, dev((j % b.page).astype(np.int64))] = dev(np.asarray(codes))[:, None, None].to(b.cache.k.dtype)


def _flat(cap, new, cached, d, keys, seed=8):
    """A batch whose products are small = 0.27 cap (rounded) times the values `keys` of the keys."""
    b = Batch(new, cached, 4, 1, d, 16, "bf16", seed=seed)
    b.q[:] = oracle.bf16_round(np.array([0.27 * cap / (d * b.scale)], np.float32))[0]
    b.d_q = dev(b.q, BF)
    values = keys(np.arange(b.ctx[0]))
    _set_keys(b, 0, np.arange(b.ctx[0]), values.astype(np.float32))
    b.keys[0][:] = values[None, :, None]
    return b


@pytest.mark.parametrize("cap", [50.0, 70.0, 80.0, 88.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", ["causal", "documents", "split", "window"])
def test_small_products_that_a_row_does_not_see(form, d, cap):
    # What a row sees scores at minus the cap; beside it in the wave others see keys that score 0.27 of it, in a step that
    # is all masked for the row: 2^(-(1 + 0.26) cap log2 e) between the two is no number for caps above about 69.
    first, window = None, 0
    if form == "causal":                                      # 124 .. 127 see the keys up to 127, 128 .. 131 those behind
        b = _flat(cap, [300], [100], d, lambda j: np.where(j < 128, -16.0, 1.0))
    elif form == "documents":                                 # small keys ahead of every other row's document
        b = _flat(cap, [300], [100], d, lambda j: np.where(j < 128, 1.0, -16.0))
        first = np.where((np.arange(300) % 2 == 1) & (np.arange(300) >= 28), 128, 0).astype(np.int32)
    elif form == "split":                                     # whole parts of them
        b = _flat(cap, [70], [4000], d, lambda j: np.where(j < 3968, 1.0, -16.0))
        first = np.where(np.arange(70) % 2 == 1, 3968, 0).astype(np.int32)
    else:                                                     # the same edge where tiles of keys begin at 96
        b = _flat(cap, [300], [100], d, lambda j: np.where(j < 224, -16.0, 1.0))
        window = 64
    b.check(b.run(window, _scores(cap, first=first)), window, f"{form} {cap}", cap=cap, first=first)


@pytest.mark.parametrize("cap", [30.0, 88.0, 89.0])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_at_the_end_of_the_polynomial(cap, sign):
    # all products of one size, 0.27 of the cap, or beyond it
    for of in (1.0, 1.04, 1.3):
        for new, cached in (([300], [200]), ([70], [2500]), ([1], [900])):
            b = _flat(cap, new, cached, 128, lambda j: np.where(j % 7 == 3, -sign * of, sign * of))
            b.check(b.run(scores=_scores(cap)), 0, f"{cap} {sign} {of} {new}", cap=cap)
