"""GPU parity of the INT8 cache (one scale for 16 rows of a kv head): codes and scales bit for bit against the
oracle where rows are written as they are, rotated keys within their rounding, rows read back, and attention.

A rotated key is off from binary64 by (2 pi 2^-26 + 2^-23 + 4 * 2^-24) (|x0| + |x1|), less than 2^-21 of the
row's largest pair's sum: its code's value is within half a step and that (twice: the step is off by as much)
of the exact value.
"""

import numpy as np
import pytest
import torch

import dequant_gemv_w4_amd as w4
import oracle
from _batch import BF, DEV, Batch, dev
from _util import to_np32

pytestmark = pytest.mark.gpu
F32 = torch.float32


def _say(*what):
    print(*what, flush=True)


class Cache:
    """An INT8 cache on the GPU and the oracle's copy."""

    def __init__(self, pages, kv, page, d, seed=0):
        rng = np.random.default_rng(seed)
        self.page, self.kv, self.d = page, kv, d
        self.codes = {n: rng.integers(-128, 128, (pages, kv, page, d)).astype(np.int8) for n in "kv"}
        self.scales = {n: np.full((pages, kv, page // 16), np.nan, np.float32) for n in "kv"}
        self.gpu = w4.W4KVCache(*(dev(self.codes[n]) for n in "kv"), *(dev(self.scales[n]) for n in "kv"))

    def write(self, x, heads, slots):
        """The oracle's write of x [T, heads + 2 kv, d]; the status bits."""
        st = 0
        for i, n in enumerate("kv"):
            st |= oracle.write_rows_ref(self.codes[n], self.scales[n], x[:, heads + i * self.kv: heads + (i + 1) * self.kv], slots)
        return st

    def same(self, what):
        for n, c, s in (("k", self.gpu.k, self.gpu.k_scales), ("v", self.gpu.v, self.gpu.v_scales)):
            bad = np.argwhere(c.cpu().numpy() != self.codes[n])
            assert bad.size == 0, f"{what} {n}: {len(bad)} codes differ, first at {bad[0]}"
            assert np.array_equal(s.cpu().numpy(), self.scales[n], equal_nan=True), f"{what} {n}: scales differ"


def _slots(table, start, n, page):
    pos = np.arange(start, start + n)
    return table[pos // page] * page + pos % page


def _rows(rng, T, width, dtype, spread=1.0):
    x = (rng.standard_normal((T, width)) * np.exp(rng.uniform(-spread, spread, (T, 1)))).astype(np.float32)
    x[:, rng.random(width) < 0.02] *= 20
    return to_np32(dev(x, dtype)) if dtype == BF else x


WRITE = [  # heads, kv, d, page, dtype, steps of new tokens per request
    (1, 1, 64, 16, F32, [[1], [1], [1]]),
    (4, 2, 128, 16, BF, [[5], [1], [16], [1], [33]]),
    (8, 8, 64, 32, F32, [[3, 40], [1, 1], [1, 1], [0, 7]]),
    (6, 3, 128, 64, BF, [[100, 1, 17], [1, 1, 1], [2, 0, 31]]),
    (0, 5, 128, 16, F32, [[20, 4], [1, 13]]),
    (0, 1, 64, 128, BF, [[15], [1], [1], [200]]),
    (33, 33, 64, 16, F32, [[9], [8]]),
    (32, 4, 128, 4096, BF, [[1, 300], [70, 1]]),
]


@pytest.mark.parametrize("case", WRITE)
def test_write_is_the_oracles(case):
    heads, kv, d, page, dtype, steps = case
    _say("write", case)
    rng = np.random.default_rng(len(steps) + kv)
    B = len(steps[0])
    total = [sum(s[b] for s in steps) for b in range(B)]
    need = [-(-t // page) for t in total]
    c = Cache(sum(need) + 1, kv, page, d, seed=kv)
    order = rng.permutation(sum(need) + 1)
    tables, used = [], 0
    for n in need:
        tables.append(order[used: used + n])
        used += n
    have = [0] * B
    for step in steps:
        slots = np.concatenate([_slots(t, h, n, page) for t, h, n in zip(tables, have, step)]).astype(np.int64)
        have = [h + n for h, n in zip(have, step)]
        x = _rows(rng, len(slots), (heads + 2 * kv) * d, dtype)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        q = w4.w4_cache_write(dev(x, dtype), c.gpu, dev(slots), status=st)
        x3 = x.reshape(len(slots), heads + 2 * kv, d)
        assert int(st) == c.write(x3, heads, slots) == 0
        c.same(str(step))
        if heads:
            assert np.array_equal(to_np32(q), oracle.bf16_round(x3[:, :heads]))
        else:
            assert q is None


def test_write_order_within_a_block_and_padding():
    # rows of a block in any order, tokens without a slot between requests, slots past the cache
    kv, d, page = 2, 64, 32
    rng = np.random.default_rng(1)
    c = Cache(4, kv, page, d)
    slots = np.array([3, 1, 2, 0, -1, 47, 40, 33, -7, 64 + 5, 128, 1 << 40, -1, 96, 97], np.int64)
    x = _rows(rng, len(slots), (4 + 2 * kv) * d, F32)
    q = torch.full((len(slots), 4, d), 7.0, dtype=BF, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    w4.w4_cache_write(dev(x), c.gpu, dev(slots), q=q, status=st)
    assert c.write(x.reshape(len(slots), -1, d), 4, slots) == 8 and int(st) == 8
    c.same("order")
    q = to_np32(q)
    for t, s in enumerate(slots):
        if s < 0 or s >= 4 * page:
            assert np.all(q[t] == 7.0), t
        else:
            assert np.array_equal(q[t], oracle.bf16_round(x[t].reshape(-1, d)[:4])), t


def test_write_of_values_and_scales_out_of_range():
    kv, d, page = 2, 128, 16
    rng = np.random.default_rng(3)
    for old in (np.nan, np.inf, -1.0, 0.0, 1e-38, 2.0 ** -100, 3e38, 1e-3, 1.0):
        for rows in ([5], [0], list(range(16)), [3, 4, 15]):
            for scale in (1.0, 0.0, 1e-30, 2.0 ** -94, 1e-40, 1e38, 2.0 ** 127):
                c = Cache(1, kv, page, d, seed=len(rows))
                for n, s in (("k", c.gpu.k_scales), ("v", c.gpu.v_scales)):
                    c.scales[n][:] = old
                    s.fill_(old)
                x = (rng.uniform(-1, 1, (len(rows), 2 * kv * d)) * scale).astype(np.float32)
                x[0, 3] = [np.nan, np.inf, -np.inf, 0.5][len(rows) % 4] if scale == 1.0 else x[0, 3]
                st = torch.zeros(1, dtype=torch.int32, device=DEV)
                w4.w4_cache_write(dev(x), c.gpu, dev(np.array(rows, np.int64)), status=st)
                assert int(st) == c.write(x.reshape(len(rows), -1, d), 0, rows), (old, rows, scale)
                c.same(f"old {old} rows {rows} scale {scale}")


@pytest.mark.parametrize("heads,kv,d,rot,inter,page,dtype", [(8, 2, 128, 128, False, 16, F32), (4, 4, 64, 32, True, 32, BF),
                                                             (5, 1, 128, 48, False, 64, BF), (16, 16, 64, 64, True, 16, F32)])
def test_rope_write(heads, kv, d, rot, inter, page, dtype):
    _say("rope", heads, kv, d, rot, inter, page)
    rng = np.random.default_rng(rot)
    new, cached = [1, 40, 3, 16], [700000, 0, 1000, 32]
    pages, slots, pos = 0, [], []
    for n, at in zip(new, cached):
        first = at % 16
        slots.append(pages * page + first + np.arange(n))
        pos.append(at + np.arange(n))
        pages += -(-(first + n) // page)
    slots, pos = np.concatenate(slots).astype(np.int64), np.concatenate(pos).astype(np.int32)
    T = len(slots)
    x = _rows(rng, T, (heads + 2 * kv) * d, dtype, 0.3)
    c = Cache(pages + 1, kv, page, d)
    for n, s in (("k", c.gpu.k_scales), ("v", c.gpu.v_scales)):
        c.scales[n][:] = 0.3
        s.fill_(0.3)
    before = {n: oracle.block_values(c.codes[n], c.scales[n]) for n in "kv"}
    rope = w4.W4Rope.make(rot, 10000.0, inter)
    freqs, _ = w4.w4_rope_frequencies(rope, DEV)
    q = w4.w4_rope_cache(dev(x, dtype), c.gpu, dev(pos), dev(slots), rope, freqs)
    # q as beside a bfloat16 cache
    other = w4.W4KVCache.empty(pages + 1, page, kv, d, device=DEV)
    assert torch.equal(q, w4.w4_rope_cache(dev(x, dtype), other, dev(pos), dev(slots), rope, freqs))
    x3 = x.reshape(T, -1, d)
    ref_f, amp = oracle.rope_frequencies_ref(rot, 10000.0)
    turned = oracle.rope_ref(x3[:, : heads + kv], pos, ref_f, amp, inter)
    # V: bit for bit
    oracle.write_rows_ref(c.codes["v"], c.scales["v"], x3[:, heads + kv:], slots)
    assert np.array_equal(c.gpu.v.cpu().numpy(), c.codes["v"]) and np.array_equal(c.gpu.v_scales.cpu().numpy(), c.scales["v"])
    # K: the scale and the values within the rotation's rounding
    ref = dict(codes=c.codes["k"].copy(), scales=c.scales["k"].copy())
    oracle.write_rows_ref(ref["codes"], ref["scales"], turned[:, heads:], slots)
    got_s, got_c = c.gpu.k_scales.cpu().numpy(), c.gpu.k.cpu().numpy()
    assert np.all(np.abs(got_s - ref["scales"]) <= 2.0 ** -20 * ref["scales"])
    values = oracle.block_values(got_c, got_s)
    pg, at = slots // page, slots % page
    half = 0.5 * got_s.astype(np.float64)[pg, :, at // 16][..., None]
    off = np.abs(values[pg, :, at] - turned[:, heads:])
    assert np.all(off <= half * (1 + 2.0 ** -18) + 2.0 ** -20 * np.abs(turned[:, heads:]).max(-1, keepdims=True))
    # other rows: as they were, or rescaled once within half a step
    others = np.ones(got_c.shape, bool)
    others[pg, :, at] = False
    step = np.repeat(got_s.astype(np.float64), 16, 2)[..., None]
    new_blocks = np.zeros(got_s.shape, bool)
    first = at % 16 == 0
    new_blocks[pg[first], :, at[first] // 16] = True
    kept = others & ~np.repeat(new_blocks, 16, 2)[..., None]
    assert np.all((np.abs(values - before["k"]) <= 0.5 * step * (1 + 2.0 ** -18))[kept])
    assert np.array_equal(got_c[others & ~kept], c.codes["k"][others & ~kept])


def test_writes_of_many_tokens_and_heads():
    # more tokens than workgroups at once, kv heads past a workgroup's waves; rows behind are left
    kv, d, page, T = 12, 64, 64, 5003
    rng = np.random.default_rng(9)
    pages = -(-T // page) + 1
    c = Cache(pages, kv, page, d)
    order = rng.permutation(pages)
    slots = _slots(order, 0, T, page).astype(np.int64)
    x = _rows(rng, T, 2 * kv * d, BF)
    w4.w4_cache_write(dev(x, BF), c.gpu, dev(slots))
    c.write(x.reshape(T, -1, d), 0, slots)
    c.same("many")


def test_write_graph_and_stream():
    kv, d, page = 4, 128, 16
    rng = np.random.default_rng(5)
    c = Cache(8, kv, page, d)
    x = torch.zeros(3, 2 * kv * d, dtype=F32, device=DEV)
    slots = torch.zeros(3, dtype=torch.int64, device=DEV)
    w4.w4_cache_write(x, c.gpu, slots.fill_(-1))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.w4_cache_write(x, c.gpu, slots)
    side = torch.cuda.Stream()
    for i in range(40):                                       # three requests, a token each a step
        s = np.array([i % 32, 32 + (i + 5) % 32, -1 if i % 3 else 64 + i], np.int64)
        rows = _rows(rng, 3, 2 * kv * d, F32)
        x.copy_(dev(rows))
        slots.copy_(dev(s))
        torch.cuda.synchronize()
        if i % 4 == 3:
            with torch.cuda.stream(side):
                w4.w4_cache_write(x, c.gpu, slots)
        else:
            g.replay()
        torch.cuda.synchronize()
        c.write(rows.reshape(3, -1, d), 0, s)
        if i % 8 == 7:
            c.same(f"step {i}")


# --------------------------------------------------------------------------
# Rows read back
# --------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("n,kv,d,page,dtype", [(1, 1, 64, 16, BF), (7, 3, 128, 32, F32), (130, 2, 64, 64, BF), (1000, 5, 128, 16, F32),
                                               (3, 33, 64, 4096, BF), (4099, 1, 128, 128, BF)])
def test_read(kind, n, kv, d, page, dtype):
    _say("read", kind, n, kv, d, page)
    b = Batch([1], [n], kv, kv, d, page, kind, seed=n)
    slots = _slots(b.table[0], 0, n, page).astype(np.int64)
    out = w4.w4_cache_read(b.cache, dev(slots), out_dtype=dtype)
    ref = np.concatenate([b.keys[0][:, :n], b.values[0][:, :n]]).transpose(1, 0, 2).reshape(n, -1)
    ref32 = ref.astype(np.float32)                            # code * scale: 8 and 24 bits, one rounding
    assert np.array_equal(to_np32(out), oracle.bf16_round(ref32) if dtype == BF else ref32)


def test_read_slots_repeated_left_out_and_past():
    kv, d, page = 2, 64, 16
    b = Batch([1], [40], kv, kv, d, page, "int8", seed=2)
    slots = _slots(b.table[0], 0, 41, page).astype(np.int64)
    pick = np.array([5, 5, 0, 40, 17, 5])
    s = slots[pick].copy()
    s[1], s[4] = -1, b.cache.pages * page
    out = torch.full((6, 2 * kv * d), 7.0, dtype=F32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert w4.w4_cache_read(b.cache, dev(s), out=out, status=st) is out
    assert int(st) == 8
    ref = np.concatenate([b.keys[0], b.values[0]]).transpose(1, 0, 2).reshape(41, -1)[pick].astype(np.float32)
    ref[[1, 4]] = 7.0
    assert np.array_equal(to_np32(out), ref)
    st.zero_()
    w4.w4_cache_read(b.cache, torch.full((9,), -1, dtype=torch.int64, device=DEV), status=st)
    assert int(st) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_read_and_write_into_another_cache(d):
    # whole blocks that no row has outgrown come back as the same codes, by way of binary32 rows
    kv, page = 3, 32
    a, b = w4.W4KVCache.empty(6, page, kv, d, int8=True, device=DEV), w4.W4KVCache.empty(6, 16, kv, d, int8=True, device=DEV)
    x = torch.randn(80, 2 * kv * d, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    slots_a, slots_b = torch.arange(80, device=DEV) + 64, torch.arange(80, device=DEV) + 16
    w4.w4_cache_write(x, a, slots_a)
    rows = w4.w4_cache_read(a, slots_a, out_dtype=F32)
    assert w4.w4_cache_write(rows, b, slots_b) is None
    assert torch.equal(w4.w4_cache_read(b, slots_b, out_dtype=BF), w4.w4_cache_read(a, slots_a))
    ka, kb = (c.k.permute(0, 2, 1, 3).reshape(-1, kv, d)[s] for c, s in ((a, slots_a), (b, slots_b)))
    assert torch.equal(ka, kb)
    # and through a bfloat16 cache: its rows are the values rounded
    c = w4.W4KVCache.empty(6, 16, kv, d, device=DEV)
    w4.w4_cache_write(rows, c, slots_b)
    assert torch.equal(w4.w4_cache_read(c, slots_b), rows.to(BF))


def test_far_offsets():
    # codes past 2^32 bytes, written, read and attended
    pages, page, kv, d = 540_000, 16, 8, 64
    c = w4.W4KVCache.empty(pages, page, kv, d, int8=True, device=DEV)
    assert c.k.numel() > 2 ** 32
    at = (pages - 2) * page + 3
    slots = torch.tensor([at, at + 1, 7], device=DEV)
    x = torch.arange(3 * 2 * kv * d, device=DEV, dtype=F32).view(3, -1).remainder(127.0)
    w4.w4_cache_write(x, c, slots)
    assert bool((w4.w4_cache_read(c, slots, out_dtype=F32) - x).abs().max() <= 1.0 / 2)
    far = (pages - 1) * page
    v = torch.full((16, 2 * kv * d), 3.0, device=DEV)
    w4.w4_cache_write(v, c, torch.arange(far, far + 16, device=DEV))
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV)
    o = w4.w4_paged_attention(torch.zeros(1, kv, d, dtype=BF, device=DEV), c, table, torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                              torch.tensor([16], dtype=torch.int32, device=DEV), 1.0)
    assert bool((o == 3.0).all())


# --------------------------------------------------------------------------
# Attention over an INT8 cache
# --------------------------------------------------------------------------

ATTEND = [  # new, cached, heads, kv, d, page, window
    ([1], [0], 1, 1, 64, 16, 0),
    ([1], [15], 8, 8, 128, 16, 0),
    ([1], [16], 4, 1, 64, 16, 0),
    ([1], [33], 40, 1, 128, 32, 0),
    ([1], [1000], 32, 8, 64, 16, 0),
    ([1], [20001], 8, 1, 128, 64, 0),
    ([1] * 7, [0, 1, 30, 31, 32, 500, 3001], 12, 4, 128, 16, 0),
    ([3, 0, 4, 1], [5, 9, 60, 700], 8, 1, 128, 16, 0),
    ([5, 1, 0, 40], [0, 100, 3, 77], 8, 1, 64, 32, 0),
    ([33], [0], 4, 4, 64, 16, 0),
    ([300], [0], 4, 4, 128, 32, 0),
    ([257], [1000], 6, 2, 64, 64, 0),
    ([130, 1, 70, 1, 1], [500, 2000, 0, 63, 64], 16, 2, 128, 16, 0),
    ([600], [5000], 8, 1, 128, 128, 0),
    ([1] * 4, [200, 5, 700, 64], 8, 2, 128, 16, 64),
    ([200, 3], [100, 400], 4, 2, 128, 16, 33),
    ([64, 64], [0, 64], 5, 5, 128, 16, 1),
    ([1] * 2, [700, 9000], 40, 1, 64, 4096, 100),
    ([6, 0, 0, 3, 0], [100, 5, 6, 50, 2], 8, 1, 128, 16, 0),
    ([6, 1, 8, 30, 5], [3000, 900, 40, 7, 1000], 16, 2, 128, 16, 0),
]


@pytest.mark.parametrize("case", ATTEND)
def test_attention(case):
    new, cached, heads, kv, d, page, window = case
    _say("int8 attention", case)
    b = Batch(new, cached, heads, kv, d, page, "int8", seed=len(new) + heads, pad=3, wide=2)
    b.check(b.run(window), window, str(case))


@pytest.mark.parametrize("new,cached", [([1, 1], [300, 70]), ([90, 3], [110, 50])])
def test_attention_keeps_masked_scales_out(new, cached):
    # a scale that is not finite reaches the rows that see its block and no other
    for which in "kv":
        b = Batch(new, cached, 4, 2, 128, 16, "int8", seed=5)
        clean = to_np32(b.run())
        b.check(b.run(), 0, "clean")
        j = (b.ctx[0] - 1) // 16 * 16                         # the last block of the first request
        getattr(b.cache, which + "_scales")[int(b.table[0, j // 16]), :, 0] = float("nan")
        got = to_np32(b.run())
        for t in range(new[0]):
            row, was = got[t], clean[t]
            if b.ctx[0] - new[0] + t >= j:
                assert np.isnan(row).any(), t
            else:
                assert np.all(np.abs(row - was) <= 4 * 2.0 ** -8 * np.abs(was) + 0.02), t
        s = slice(new[0], new[0] + new[1])
        assert np.all(np.abs(got[s] - clean[s]) <= 4 * 2.0 ** -8 * np.abs(clean[s]) + 0.02)


def test_attention_bad_pages_read_as_zeros():
    for new, cached in (([1], [199]), ([90], [110])):
        b = Batch(new, cached, 4, 2, 64, 16, "int8", seed=6)
        for entry, value in ((2, -1), (5, b.cache.pages), (7, 2 ** 31 - 1), (9, -(2 ** 31))):
            b.table[0, entry] = value
            for x in (b.keys[0], b.values[0]):
                x[:, entry * 16: entry * 16 + 16] = 0.0
        b.d_table = dev(b.table)
        b.check(b.run(), 0, "bad pages", status=8)


# --------------------------------------------------------------------------
# A run of the operators, and refusals that need device tensors
# --------------------------------------------------------------------------

def test_a_request_from_write_to_attention():
    # a prompt and then single tokens: tables, write, attention; and the cache read back is what was attended
    heads, kv, d, page, B = 8, 2, 64, 16, 3
    rng = np.random.default_rng(4)
    cache = w4.W4KVCache.empty(40, page, kv, d, int8=True, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    lens, free, count = torch.zeros(B, **i32), torch.arange(40, **i32), torch.full((1,), 40, **i32)
    table = torch.full((B, 10), -1, **i32)
    for new in ([37, 5, 60], [1, 1, 1], [1, 1, 1], [3, 0, 20]):
        T = sum(new) + 2
        cu, pos, slots = w4.w4_block_tables(torch.tensor(new, **i32), lens, free, count, table, page, tokens=T)
        x = dev(_rows(rng, T, (heads + 2 * kv) * d, F32, 0.3), BF)
        q = w4.w4_cache_write(x, cache, slots)
        o = to_np32(w4.w4_paged_attention(q, cache, table, cu, lens, d ** -0.5))
        start = 0
        for b, n in enumerate(new):
            ctx = int(lens[b])
            at = torch.arange(ctx, device=DEV)
            rows = to_np32(w4.w4_cache_read(cache, table[b].long()[at // page] * page + at % page, out_dtype=F32)).reshape(ctx, 2, kv, d)
            if n:
                ref, w = oracle.attention_ref(to_np32(q)[start: start + n], rows[:, 0].transpose(1, 0, 2), rows[:, 1].transpose(1, 0, 2), ctx, d ** -0.5)
                assert np.all(np.abs(o[start: start + n] - ref) <= (2.0 ** -8 + 2.0 ** -12) * w + 2.0 ** -8 * np.abs(ref))
            start += n


def test_python_layer_refusals():
    c = w4.W4KVCache.empty(2, 32, 1, 64, device=DEV, int8=True)
    assert c.k.dtype == torch.int8 and tuple(c.k_scales.shape) == (2, 1, 2)
    with pytest.raises(TypeError):
        w4.W4KVCache(c.k, c.v)                                # no scales
    with pytest.raises(ValueError):
        w4.W4KVCache(c.k, c.v, torch.ones(2, 1, 32, device=DEV), torch.ones(2, 1, 32, device=DEV))   # a scale a row
    with pytest.raises(TypeError):
        w4.W4KVCache(c.k, c.v.view(torch.uint8), c.k_scales, c.v_scales)
    with pytest.raises(ValueError):
        w4.W4KVCache.empty(2, 32, 1, 64, fp8=True, int8=True, device=DEV)
    slots = torch.zeros(3, dtype=torch.int64, device=DEV)
    x = torch.zeros(3, 128, device=DEV)
    with pytest.raises(ValueError):
        w4.w4_cache_write(x, c, slots, q=torch.zeros(3, 1, 64, dtype=BF, device=DEV))
    with pytest.raises(ValueError):
        w4.w4_cache_write(x[:, :64].contiguous(), c, slots)   # fewer heads than K and V
    with pytest.raises(ValueError):
        w4.w4_cache_write(x, c, slots[:2])
    with pytest.raises(TypeError):
        w4.w4_cache_write(x, c, slots.int())
    with pytest.raises(ValueError):
        w4.w4_cache_write(x.cpu(), c, slots)
    with pytest.raises(ValueError):
        w4.w4_cache_write(torch.zeros(3, 256, device=DEV)[:, ::2], c, slots)
    with pytest.raises(ValueError):
        w4.w4_cache_read(c, slots[:, None])
    with pytest.raises(ValueError):
        w4.w4_cache_read(c, slots, out=torch.zeros(3, 64, device=DEV))
    with pytest.raises(TypeError):
        w4.w4_cache_read(c, slots, out_dtype=torch.float16)
    with pytest.raises(w4.W4Error):
        w4.w4_cache_read(c, slots[:0])                        # no rows
