"""GPU parity of attention with capped scores, a bias by distance, a document mask or a prefix mask against the
binary64 oracle (tolerances: _batch.Batch.check).
"""

import numpy as np
import pytest
import torch

import dequant_gemv_w4_amd as w4
import oracle
from _batch import BF, DEV, Batch, dev
from _util import to_np32

pytestmark = pytest.mark.gpu
UB = 2.0 ** -8


def _say(*what):
    print(*what, flush=True)


def _documents(rng, b, most):
    """First keys [rows of q]: documents of up to `most` tokens; rows of no request get values that would fault."""
    out = np.full(b.q.shape[0], 2 ** 31 - 1, np.int32)
    for i, (n, c) in enumerate(zip(b.new, b.ctx)):
        starts = [0]
        while starts[-1] < c:
            starts.append(starts[-1] + int(rng.integers(1, most + 1)))
        pos = np.arange(c - n, c)
        out[int(b.cu[i]): int(b.cu[i]) + n] = np.array(starts)[np.searchsorted(starts, pos, side="right") - 1]
    return out


def _slopes(heads):
    return (2.0 ** (-8.0 * np.arange(1, heads + 1) / heads)).astype(np.float32)


def _scores(cap=0.0, slopes=None, first=None, prefix=None):
    return w4.W4Scores(cap=cap, slopes=None if slopes is None else dev(slopes), first_keys=None if first is None else dev(first),
                       prefix_lens=None if prefix is None else dev(prefix))


CASES = [  # new, cached, heads, kv, d, page, window
    ([1], [0], 1, 1, 64, 16, 0),
    ([1], [31], 32, 1, 64, 32, 0),
    ([1], [1000], 8, 8, 128, 16, 0),
    ([1], [20001], 4, 1, 128, 64, 0),
    ([1] * 6, [0, 1, 30, 32, 500, 3001], 12, 4, 128, 16, 0),
    ([1] * 4, [200, 5, 700, 64], 8, 2, 128, 16, 64),
    ([1] * 9, [2500, 1, 300, 0, 31, 1500, 63, 64, 90], 32, 1, 64, 16, 0),     # 32 rows a tile
    ([3, 0, 4, 1], [5, 9, 60, 700], 8, 1, 128, 16, 0),
    ([6, 0, 0, 3, 0], [100, 5, 6, 50, 2], 8, 1, 64, 16, 0),                   # as many tokens as requests, not one each
    ([5, 1, 0, 40], [0, 100, 3, 77], 8, 1, 128, 32, 0),
    ([33], [0], 4, 4, 64, 16, 0),
    ([300], [0], 4, 4, 128, 32, 0),
    ([257], [900], 3, 1, 64, 64, 0),
    ([130, 1, 70, 1, 1], [500, 2000, 0, 63, 64], 4, 1, 128, 16, 0),
    ([300], [2500], 4, 1, 128, 128, 0),                                       # few tiles over many keys: split
    ([200, 3], [100, 400], 4, 2, 128, 16, 33),
    ([6, 1, 8, 30, 5], [1500, 900, 40, 7, 1000], 16, 2, 64, 16, 0),           # 48, 8, 64, 240 and 40 rows
]
FORMS = ["cap", "slopes", "docs", "prefix", "all"]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("form", FORMS)
def test_scores(form, kind):
    rng = np.random.default_rng(FORMS.index(form))
    for i, case in enumerate(CASES):
        new, cached, heads, kv, d, page, window = case
        if (i + FORMS.index(form) + len(kind)) % 2 and i > 6:                 # every other of the longer ones
            continue
        _say(form, kind, case)
        # scores around a cap: well below it, at it and far above
        qscale = [0.3, 3.0, 30.0][i % 3] if form in ("cap", "all") else 1.0
        b = Batch(new, cached, heads, kv, d, page, kind, seed=i + heads, pad=3, wide=2, qscale=qscale)
        given = {}
        if form in ("cap", "all"):
            given["cap"] = [2.0, 50.0, 30.0][(i // 3) % 3]
        if form in ("slopes", "all"):
            given["slopes"] = _slopes(heads)
        if form in ("docs", "all"):
            given["first"] = _documents(rng, b, [3, 50, 700][i % 3])
        if form in ("prefix", "all"):
            given["prefix"] = rng.integers(0, np.maximum(np.array(b.ctx) + 2, 2)).astype(np.int32)
        b.check(b.run(window, _scores(**given)), window, f"{form} {kind} {case}", **given)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("new,cached", [([1, 1, 1], [40, 3000, 0]), ([150, 2], [20, 700])])
def test_record_of_zeros_is_the_plain_form(kind, new, cached):
    b = Batch(new, cached, 8, 2, 128, 16, kind, seed=1)
    plain = b.run()
    assert torch.equal(plain, b.run(scores=w4.W4Scores()))
    # slopes of zero, documents from the first token and prefixes of nothing: the same keys and scores
    zero = _scores(slopes=np.zeros(8, np.float32), first=np.zeros(b.q.shape[0], np.int32), prefix=np.zeros(len(new), np.int32))
    got, was = to_np32(b.run(scores=zero)), to_np32(plain)
    b.check(b.run(scores=zero), 0, "zeros")
    assert np.all(np.abs(got - was) <= 4 * UB * np.abs(was) + 0.01)


@pytest.mark.parametrize("cap", [2.0 ** -18, 0.01, 1.0, 88.0, 5000.0, 80000.0])
def test_caps_over_the_range(cap):
    # caps far below, at and far above the scores; the largest and smallest that the scale (2^-3.5) allows
    for new, cached in (([1], [700]), ([70], [60])):
        for qscale in (0.05, 1.0, 60.0):
            b = Batch(new, cached, 4, 2, 128, 16, "bf16", seed=3, qscale=qscale)
            b.check(b.run(scores=w4.W4Scores(cap=cap)), 0, f"cap {cap} {qscale}", cap=cap)


@pytest.mark.parametrize("cap", [30.0, 88.0, 89.0])
@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 64), ("int8", 128)])
def test_capped_scores_far_below_zero(cap, kind, d):
    # every key against the query, at not quite a quarter of the cap, and one along it that only the last token sees
    for new, cached in (([300], [200]), ([300], [2500]), ([1], [900])):
        b = Batch(new, cached, 4, 1, d, 16, kind, seed=8)
        x = float(oracle.bf16_round(np.array([0.24 * cap / (d * b.scale)], np.float32))[0])
        b.q[:] = -x
        b.d_q = dev(b.q, BF)
        last, one = b.ctx[0] - 1, 1.0 if kind == "bf16" else 127.0
        b.cache.k.fill_(int(one) if kind == "int8" else one)
        b.cache.k[int(b.table[0, last // 16]), :, last % 16] = -int(one) if kind == "int8" else -one
        if kind == "int8":
            b.cache.k_scales.fill_(1.0 / 128)
        b.keys[0][:] = one if kind == "bf16" else one / 128
        b.keys[0][:, last] *= -1
        b.check(b.run(scores=w4.W4Scores(cap=cap)), 0, f"{cap} {kind} {new} {cached}", cap=cap)


def test_slopes_negative_large_and_far():
    # a bias that grows with the distance, one that leaves the row's own key alone, and distances past 2^16
    for new, cached in (([1], [70000]), ([40], [300])):
        b = Batch(new, cached, 4, 1, 64, 64, "bf16", seed=5)
        for slopes in ([-0.01, 0.0, 1000.0, 1e-6], [3e4, -1e-3, 0.5, 0.25]):
            s = np.array(slopes, np.float32)
            b.check(b.run(scores=_scores(slopes=s)), 0, f"slopes {slopes}", slopes=s)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("new,cached,window", [([4, 1, 1], [60, 900, 10], 0), ([90, 40], [30, 500], 0), ([1, 1], [300, 40], 64), ([90], [200], 50)])
def test_ranges_of_any_values(kind, new, cached, window):
    # rows that see nothing, documents that begin behind the row, prefixes past the end, numbers at the ends of int32
    b = Batch(new, cached, 8, 2, 64, 16, kind, seed=8, pad=2)
    rng = np.random.default_rng(9)
    T = b.q.shape[0]
    ends = np.array([-(2 ** 31), -1, 0, 1, 16, 2 ** 30, 2 ** 31 - 1])
    for trial in range(6):
        first = np.where(rng.random(T) < 0.4, rng.choice(ends, T), rng.integers(0, max(b.ctx) + 3, T)).astype(np.int32)
        prefix = np.where(rng.random(len(new)) < 0.4, rng.choice(ends, len(new)), rng.integers(0, max(b.ctx) + 3, len(new))).astype(np.int32)
        for given in (dict(first=first), dict(prefix=prefix), dict(first=first, prefix=prefix), dict(first=first, slopes=_slopes(8), cap=5.0)):
            got = b.run(window, _scores(**given))
            b.check(got, window, f"{trial} {sorted(given)}", **given)
    none = np.full(T, 2 ** 30, np.int32)
    got = to_np32(b.run(window, _scores(first=none)))
    assert np.all(got[: int(b.cu[-1])] == 0) and np.all(got[int(b.cu[-1]):] == 7.0)


def test_short_lengths_with_a_prefix():
    # lens below the new tokens: the first rows have no position, but see the prefix as far as there are keys
    b = Batch([4, 3], [60, 20], 8, 2, 64, 16, "bf16", seed=4, pad=2)
    b.d_lens = dev(np.array([2, 0], np.int32))
    got = to_np32(b.run(scores=_scores(prefix=np.array([50, 50], np.int32))))
    ref, w = oracle.attention_scores_ref(b.q[:4], b.keys[0][:, :2], b.values[0][:, :2], 2, b.scale, prefix=50)
    assert np.all(np.abs(got[:4] - ref) <= (UB + 1e-4) * w + UB * np.abs(ref))
    assert np.all(got[4:7] == 0) and np.all(got[7:] == 7.0)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("new,cached", [([40], [100]), ([3, 50, 1], [10, 0, 800]), ([1, 1], [3000, 70])])
@pytest.mark.parametrize("form", ["docs", "prefix", "cap", "slopes"])
def test_masked_keys_stay_out(kind, new, cached, form):
    # an infinity or NaN at a key reaches the rows that see the key and no other
    rng = np.random.default_rng(2)
    b = Batch(new, cached, 8, 2, 128, 16, kind, seed=21)
    given = dict(docs=lambda: dict(first=_documents(rng, b, 30)), prefix=lambda: dict(prefix=np.array([c // 2 for c in b.ctx], np.int32)),
                 cap=lambda: dict(cap=30.0), slopes=lambda: dict(slopes=_slopes(8)))[form]()
    scores = _scores(**given)
    clean = to_np32(b.run(scores=scores))
    b.check(b.run(scores=scores), 0, "clean", **given)
    for which, value in (("v", float("nan")), ("v", float("inf")), ("k", float("nan"))):
        c = Batch(new, cached, 8, 2, 128, 16, kind, seed=21)
        hit = [max(0, n_c - 1 - (n > 2) * 7) for n, n_c in zip(new, c.ctx)]
        for i, j in enumerate(hit):
            page = int(c.table[i, j // 16])
            row = getattr(c.cache, which)[page, :, j % 16]
            if kind == "fp8":
                row[:, 5] = 0x7F
                if value == float("inf"):
                    getattr(c.cache, which + "_scales")[page, :, j % 16] = float("inf")
            else:
                row[:, 5] = value
        got = to_np32(c.run(scores=scores))
        for i, (j, n) in enumerate(zip(hit, new)):
            for t in range(n):
                r = int(c.cu[i]) + t
                lo, hi = oracle.key_range_ref(c.ctx[i] - n + t, c.ctx[i], 0, int(given["first"][r]) if "first" in given else None,
                                              int(given["prefix"][i]) if "prefix" in given else None)
                row, was = got[r], clean[r]
                if lo <= j <= hi:
                    # a weight that the bias has made zero leaves nothing of an infinity: heads of small slopes keep it
                    assert not np.isfinite(row[-1, 5]), (which, value, i, t)
                    if which == "k":
                        assert np.isnan(row[-1]).all()
                else:
                    assert np.all(np.abs(row - was) <= 4 * UB * np.abs(was) + 0.02), (which, value, i, t)


def test_pages_outside_the_ranges_are_not_looked_up():
    # pages ahead of every row's document, given back: no status, right results
    for new, cached in (([1], [900]), ([60], [900])):
        for kind in ("bf16", "int8"):
            b = Batch(new, cached, 8, 2, 128, 16, kind, seed=13)
            first = np.full(b.q.shape[0], 500, np.int32)
            b.table[0, : 500 // 16] = -1
            b.d_table = dev(b.table)
            b.check(b.run(scores=_scores(first=first)), 0, "given back", first=first)
            b.table[0, 500 // 16 + 3] = -1                    # one that is seen
            b.d_table = dev(b.table)
            at = (500 // 16 + 3) * 16
            for x in (b.keys[0], b.values[0]):
                x[:, at: at + 16] = 0.0
            for given in (dict(first=first), dict(first=first, slopes=_slopes(8)), dict(first=first, cap=20.0)):
                b.check(b.run(scores=_scores(**given)), 0, f"missing {sorted(given)}", status=8, **given)


@pytest.mark.parametrize("new,cached", [([1] * 3, [3000, 40, 900]), ([70, 1, 4], [2000, 300, 5])])
def test_graph_and_streams(new, cached):
    b = Batch(new, cached, 16, 2, 128, 16, "bf16", seed=8)
    slopes, first = dev(_slopes(16)), dev(np.zeros(b.q.shape[0], np.int32))
    prefix = dev(np.array([100, 0, 3], np.int32))
    scores = w4.W4Scores(cap=30.0, slopes=slopes, first_keys=first, prefix_lens=prefix)
    ref = b.run(scores=scores)
    for _ in range(3):                                        # the same call twice is the same to the bit
        assert torch.equal(b.run(scores=scores), ref)
    bufs = [dict(o=torch.zeros_like(ref), workspace=b.workspace()) for _ in range(2)]
    call = lambda buf: w4.w4_paged_attention_scores(b.d_q, b.cache, b.d_table, b.d_cu, b.d_lens, b.scale, scores, **buf)  # noqa: E731
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(bufs[0])
    for i in range(4):                                        # other documents and prefixes in the same graph
        first.fill_(13 * i)
        prefix.fill_(50 * i)
        bufs[0]["o"].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs[0]["o"], b.run(scores=scores)), i
    first.zero_()
    prefix.copy_(dev(np.array([100, 0, 3], np.int32)))
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, buf in zip(side, bufs):                            # two calls at once, with a workspace each
        with torch.cuda.stream(s):
            for _ in range(5):
                call(buf)
    torch.cuda.synchronize()
    assert torch.equal(bufs[0]["o"], ref) and torch.equal(bufs[1]["o"], ref)


def test_python_layer_refusals():
    b = Batch([2, 1], [5, 9], 4, 2, 64, 16, "bf16")
    i32, f32 = dict(dtype=torch.int32, device=DEV), dict(dtype=torch.float32, device=DEV)
    for bad in (dict(slopes=torch.zeros(3, **f32)), dict(first_keys=torch.zeros(2, **i32)), dict(prefix_lens=torch.zeros(3, **i32)),
                dict(slopes=torch.zeros(4, 1, **f32))):
        with pytest.raises(ValueError):
            b.run(scores=w4.W4Scores(**bad))
    for bad in (dict(slopes=torch.zeros(4, dtype=torch.float64, device=DEV)), dict(first_keys=torch.zeros(3, dtype=torch.int64, device=DEV)),
                dict(prefix_lens=torch.zeros(2, **f32))):
        with pytest.raises(TypeError):
            w4.W4Scores(**bad)
    with pytest.raises(ValueError):
        w4.W4Scores(slopes=torch.zeros(8, **f32)[::2])
    for cap in (-1.0, float("nan"), 1e9):
        with pytest.raises(w4.W4Error) as e:
            b.run(scores=w4.W4Scores(cap=cap))
        assert e.value.status == 10
