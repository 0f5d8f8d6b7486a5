"""GPU parity of attention with capped or biased scores at the ends of what its steps of keys may hold, against the
binary64 oracle (tolerances: _batch.Batch.check, where no other stands at the test).
"""

import numpy as np
import pytest
import torch

import dequant_gemv_w4_amd as w4
import oracle
from _batch import BF, U32, UB, Batch, dev
from _util import to_np32

pytestmark = pytest.mark.gpu


def _scores(cap=0.0, slopes=None, first=None, prefix=None):
    return w4.W4Scores(cap=cap, slopes=None if slopes is None else dev(slopes), first_keys=None if first is None else dev(first),
                       prefix_lens=None if prefix is None else dev(prefix))


def _set_keys(b, i, j, codes):
    """Keys j of request i get the elements codes [len(j)] (of a bfloat16 cache; codes under the scales that an 8-bit one
    has), in the cache alone."""
    pg = dev(b.table[i, j // b.page].astype(np.int64))
    b.cache.k[pg, :, dev((j % b.page).astype(np.int64))] = dev(np.asarray(codes))[:, None, None].to(b.cache.k.dtype)


def _flat(cap, new, cached, d, keys, seed=8, kind="bf16"):
    """A batch whose products are 0.27 cap (rounded) times the values `keys` of the keys (E4M3: of 1, -1 and -16)."""
    b = Batch(new, cached, 4, 1, d, 16, kind, seed=seed)
    b.q[:] = oracle.bf16_round(np.array([0.27 * cap / (d * b.scale)], np.float32))[0]
    b.d_q = dev(b.q, BF)
    values = keys(np.arange(b.ctx[0]))
    codes = values.astype(np.float32)
    if kind == "fp8":
        codes = np.select([values == 1, values == -1, values == -16], [0x38, 0xB8, 0xD8]).astype(np.uint8)
        b.cache.k_scales.fill_(1.0)
    _set_keys(b, 0, np.arange(b.ctx[0]), codes)
    b.keys[0][:] = values[None, :, None]
    return b


@pytest.mark.parametrize("cap", [50.0, 70.0, 80.0, 88.0])
@pytest.mark.parametrize("kind,d", [("bf16", 64), ("bf16", 128), ("fp8", 64), ("fp8", 128)])
@pytest.mark.parametrize("form", ["causal", "documents", "split", "window"])
def test_small_products_that_a_row_does_not_see(form, kind, d, cap):
    # What a row sees scores at minus the cap; beside it in the wave others see keys that score 0.27 of it, in a step that
    # is all masked for the row: 2^(-(1 + 0.26) cap log2 e) between the two is no number for caps above about 69.
    first, window = None, 0
    if form == "causal":                                      # 124 .. 127 see the keys up to 127, 128 .. 131 those behind
        b = _flat(cap, [300], [100], d, lambda j: np.where(j < 128, -16.0, 1.0), kind=kind)
    elif form == "documents":                                 # small keys ahead of every other row's document
        b = _flat(cap, [300], [100], d, lambda j: np.where(j < 128, 1.0, -16.0), kind=kind)
        first = np.where((np.arange(300) % 2 == 1) & (np.arange(300) >= 28), 128, 0).astype(np.int32)
    elif form == "split":                                     # whole parts of them
        b = _flat(cap, [70], [4000], d, lambda j: np.where(j < 3968, 1.0, -16.0), kind=kind)
        first = np.where(np.arange(70) % 2 == 1, 3968, 0).astype(np.int32)
    else:                                                     # the same edge where tiles of keys begin at 96
        b = _flat(cap, [300], [100], d, lambda j: np.where(j < 224, -16.0, 1.0), kind=kind)
        window = 64
    b.check(b.run(window, _scores(cap, first=first)), window, f"{form} {cap}", cap=cap, first=first)


@pytest.mark.parametrize("cap", [30.0, 88.0, 89.0])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_scores_at_the_end_of_the_polynomial(kind, d, sign, cap):
    # all products of one size, 0.27 of the cap, or beyond it
    for of in (1.0, 1.04, 1.3):
        for new, cached in (([300], [200]), ([70], [2500]), ([1], [900])):
            b = _flat(cap * of, new, cached, d, lambda j: np.where(j % 7 == 3, -sign, sign), kind=kind)
            b.check(b.run(scores=_scores(cap)), 0, f"{kind} {d} {cap} {sign} {of} {new}", cap=cap)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_all_at_minus_the_polynomials_end(d, kind):
    # the maximum is taken for 36 powers of two above what every key scores
    for new, cached in (([300], [212]), ([300], [2500]), ([260], [252])):
        b = _flat(88.0, new, cached, d, lambda j: np.where(j >= 0, -1.0, 1.0), kind=kind)
        b.check(b.run(scores=_scores(88.0)), 0, f"{kind} {d} {new}", cap=88.0)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("heads", [4, 12])
@pytest.mark.parametrize("slopes", [False, True])
def test_small_scores_beside_large_ones(slopes, heads, kind):
    # One head's scores reach a cap of 60000 and more, the others' are of size 1 in the same tile.  Tolerance as in
    # _batch.Batch.check, with the size of each row's own products and weights in two bfloat16 parts (2^-16): single tokens.
    cap = 60000.0
    d, s = 128, (2.0 ** -np.arange(3, 3 + heads)).astype(np.float32) if slopes else None
    b = Batch([1] * 4, [5, 30, 40, 90], heads, 1, d, 16, kind, seed=6, qscale=1.0)
    b.q[:, 1] *= 2.0 ** 17
    b.d_q = dev(b.q, BF)
    got = to_np32(b.run(scores=_scores(cap, s))).astype(np.float64)
    for i, ctx in enumerate(b.ctx):
        ref, w = oracle.attention_scores_ref(b.q[i: i + 1], b.keys[i], b.values[i], ctx, b.scale, cap=cap, slopes=s)
        size = b.scale * np.abs(b.q[i]).sum(-1) * np.abs(b.keys[i]).max()       # [heads]
        bias = 0.0 if s is None else s * ctx
        score = (d + 4) * U32 * size + 2.0 ** -19 * size + 4 * U32 * (size + bias)
        tol = (2.0 ** -16 + 2 * (score[:, None] + (4 + ctx / 8) * U32)) * w[0] + UB * np.abs(ref[0])
        off = np.abs(got[i] - ref[0])
        worst = float(np.delete(off - tol, 1, 0).max())
        assert worst <= 0, (i, worst)
        assert np.all(np.isfinite(got[i, 1]))


@pytest.mark.parametrize("slopes", [False, True])
def test_small_scores_beside_large_ones_in_chunks(slopes):
    # Documents of two tokens with values of 1 and -1, so that the difference of their weights is what comes out: a weight
    # is off by 2^-8 and by its score's error, the sum of both by the scores'.
    cap, d, n = 90000.0, 128, 300
    s = np.array([0.125, 0.25, 0.5, 1.0], np.float32) if slopes else None
    b = Batch([n], [0], 4, 1, d, 16, "bf16", seed=7, qscale=0.1)
    b.q[:, 1] *= 2.0 ** 22
    b.d_q = dev(b.q, BF)
    j = np.arange(n)
    b.values[0][:] = np.where(j % 2, -1.0, 1.0)[None, :, None]
    b.cache.v[dev(b.table[0, j // 16].astype(np.int64)), :, dev((j % 16).astype(np.int64))] = dev(b.values[0][0].astype(np.float32), BF)[:, None]
    first = np.maximum(j - 1, 0).astype(np.int32)
    got = to_np32(b.run(scores=_scores(cap, s, first=first))).astype(np.float64)
    ref, w = oracle.attention_scores_ref(b.q, b.keys[0], b.values[0], n, b.scale, cap=cap, slopes=s, first=first)
    size = b.scale * np.abs(b.q).sum(-1) * np.abs(b.keys[0]).max()
    bias = 0.0 if s is None else s
    score = (d + 4) * U32 * size + 2.0 ** -19 * size + 4 * U32 * (size + bias)
    tol = (UB + 2 * (score[..., None] + 8 * U32)) * w + UB * np.abs(ref)
    worst = np.delete(np.abs(got - ref) - tol, 1, 1).max()
    assert worst <= 0, worst
    assert np.all(np.isfinite(got))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("new,cached", [([1], [70]), ([1, 1, 1], [70, 600, 3]), ([3, 1], [37, 2]), ([7], [100]), ([40, 150], [37, 100]), ([300], [83])])
@pytest.mark.parametrize("slopes", [False, True])
def test_keys_that_no_row_sees_change_no_bit(slopes, new, cached, kind):
    # ahead of every row's document and behind the last key: zeros there, or products far above 0.28 of the cap
    given = dict(cap=200.0, slopes=(2.0 ** -np.arange(1, 9)).astype(np.float32) if slopes else None)
    outs = []
    for code in (0.0, 112.0):                                 # 112: in bfloat16, INT8; as E4M3 code 0x70, which is 2^7
        b = Batch(new, cached, 8, 2, 128, 16, kind, seed=4, qscale=2.0)
        if kind == "int8":
            b.cache.k_scales.clamp_(min=0.05)
        first = np.zeros(b.q.shape[0], np.int32)
        for i, (n, c) in enumerate(zip(new, b.ctx)):
            at = min(c - n, 37)                               # the first key that the request's rows see
            first[int(b.cu[i]): int(b.cu[i]) + n] = at
            held = 16 * (-(-c // 16))                         # of its last page
            hidden = np.concatenate([np.arange(at), np.arange(c, held)])
            pg, row = b.table[i, hidden // 16].astype(np.int64), (hidden % 16).astype(np.int64)
            for x in (b.cache.k, b.cache.v):                  # a code of zero or of the sign of q's elements, key by key
                x[dev(pg), :, dev(row)] = 0
            if len(hidden) and code:
                q = b.q[int(b.cu[i])].reshape(2, 4, 128)[:, 0]                  # along a row's query: scores of 100 at least
                k = dev(np.sign(q) * code).to(b.cache.k.dtype) if kind != "fp8" else dev(np.where(q < 0, 0xF0, 0x70).astype(np.uint8))
                b.cache.k[dev(pg), :, dev(row)] = k[None]
            if kind == "fp8":
                for s in (b.cache.k_scales, b.cache.v_scales):
                    s[dev(pg), :, dev(row)] = 1.0
        outs.append(b.run(scores=_scores(first=first, **given)))
    assert torch.equal(outs[0], outs[1]), int((outs[0] != outs[1]).sum())


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("slope", [2.0 ** 95, 2.0 ** 100, 1e38, 3.4e38])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_slopes_at_the_end_of_binary32(cap, slope, kind):
    # a weight of 1 for the row's own key, or with the sign turned for the farthest
    for new, cached in (([1], [0]), ([1, 1], [100, 2000]), ([90, 1], [500, 3]), ([70], [2500])):
        for prefix in (False, True):
            b = Batch(new, cached, 4, 1, 64, 16, kind, seed=2)
            s = np.array([slope, -slope, 0.0, slope], np.float32)
            lens = np.zeros(len(new), np.int32) if prefix else None
            got = to_np32(b.run(scores=_scores(cap, s, prefix=lens))).astype(np.float64)
            for i, (n, c) in enumerate(zip(new, b.ctx)):
                for t in range(n):
                    row = got[int(b.cu[i]) + t]
                    for h, j in ((0, c - n + t), (1, 0), (3, c - n + t)):
                        v = b.values[i][0, j]
                        assert np.all(np.abs(row[h] - v) <= 2 * UB * np.abs(v) + 2.0 ** -100), (new, prefix, i, t, h, row[h][:4], v[:4])
                    assert np.all(np.isfinite(row))
