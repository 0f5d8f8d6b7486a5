"""GPU parity of the operators between a layer's products against the binary64 oracle.

Tolerances, with u the half step of a type (binary32 2^-24, bfloat16 2^-8, E4M3 2^-4):

* norm: y = (h * s) * w with s one rounding of a binary64 value: 3 u, 4 u allowed.
* gate: exp within 1 unit in the last place (2 u), 1 + t, the product, the quotient and the last
  product one rounding each: t enters numerator and denominator, so 2 * 2 u + 4 u; 8 u allowed.
* rotation: the turn's fraction is rounded at 2^-26 turns, sine and cosine within 2 units in the
  last place of 1 (2^-23), amplitude, two products and one sum: an angle error of 2 pi 2^-26 and
  2^-23 + 4 u on each of the two addends; (2 pi 2^-26 + 2^-23 + 4 * 2^-24) (|x0| + |x1|) amplitude.
* codes are compared bit for bit with the oracle's quantizer on the binary32 row where the row
  itself can be had, else within the half step of the code.
* attention: a weight is off by its score's error (dot product of d terms, (d + 2) u sum |q k| scale)
  plus exp2's argument and result (|z| u and 2 u) plus u of bfloat16, n weighted terms are summed
  in binary32 in chains of n / 16 products; the sum of weights likewise: with
  w = sum p |v| / sum p,  |error| <= (2^-8 + 2 (score error + 4 u + n / 8 u)) w + 2^-8 |o|.
"""

import numpy as np
import pytest
import torch

import dequant_gemv_w4_amd as w4
import oracle
from _util import to_np32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32, UB = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def _close(got, ref, tol, what):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, what
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    bad = np.abs(got - ref) > tol
    if bad.any():
        i = np.unravel_index(np.argmax(np.abs(got - ref) - tol), ref.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off; at {i}: {got[i]!r} for {ref[i]!r}, tolerance {np.broadcast_to(tol, ref.shape)[i]:.3e}")


def _say(what):
    print(what, flush=True)


# --------------------------------------------------------------------------
# Norm and gate
# --------------------------------------------------------------------------

def _rows(rows, k, seed, dtype, spread=0.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, k)) * np.exp(rng.uniform(-spread, spread, (rows, 1)))
    x[:, rng.random(k) < 0.01] *= 20
    return _dev(x.astype(np.float32), dtype)


def _codes_ref(kind, y):
    return (oracle.quantize_rows_fp8_ref if kind == "fp8" else oracle.quantize_rows_int8_ref)(y)


def _same_codes(codes, scales, y, kind, what):
    rc, rs = _codes_ref(kind, y)
    c = codes.cpu().numpy()
    bad = np.argwhere(c != rc)
    assert bad.size == 0, f"{what}: {len(bad)} codes differ, first at {bad[0]}"
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), rs.view(np.uint32)), f"{what}: scales differ"


NORM_SHAPES = [(1, 128), (3, 512), (5, 640), (1, 2048), (7, 2176), (2, 4096), (65, 8192), (1, 8192), (3, 8320), (2, 28672), (1, 32896), (2, 65536)]


@pytest.mark.parametrize("rows,k", NORM_SHAPES)
@pytest.mark.parametrize("xt,rt", [(BF, BF), (F32, BF), (BF, None), (F32, F32)])
def test_rmsnorm(rows, k, xt, rt):
    _say(f"rmsnorm {rows}x{k} {xt} {rt}")
    x = _rows(rows, k, 10 * k + rows, xt, 4.0)
    w = _dev((1 + 0.2 * np.random.default_rng(k).standard_normal(k)).astype(np.float32), BF if rows % 2 else F32)
    h = to_np32(x)
    kw = {}
    if rt is not None:
        r = _rows(rows, k, 11 * k + rows, rt)
        h = oracle.residual_sum_ref(h, to_np32(r), rt == BF)
        kw = dict(residual=r, residual_out=torch.empty_like(r))
    ref = oracle.rmsnorm_ref(h, to_np32(w), 1e-5)
    y = w4.w4_rmsnorm(x, w, 1e-5, out_dtype=F32, **kw)
    _close(to_np32(y), ref, 4 * U32 * np.abs(ref), "f32")
    if rt is not None:
        assert np.array_equal(to_np32(kw["residual_out"]), h)
    yb = w4.w4_rmsnorm(x, w, 1e-5, **kw)
    assert yb.dtype == BF and torch.equal(yb, y.to(BF))
    for kind, call in (("fp8", w4.w4_rmsnorm_fp8), ("int8", w4.w4_rmsnorm_int8)):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        codes, scales = call(x, w, 1e-5, status=st, **kw)
        _same_codes(codes, scales, to_np32(y), kind, kind)
        assert int(st) == 0
    if rt is not None:   # in place
        before = kw["residual"].clone()
        y2 = w4.w4_rmsnorm(x, w, 1e-5, residual=kw["residual"], out_dtype=F32)
        assert torch.equal(y2, y) and torch.equal(kw["residual"], kw["residual_out"]) and not torch.equal(before, kw["residual"])


def test_rmsnorm_extremes():
    k = 1024
    x = np.random.default_rng(1).standard_normal((7, k)).astype(np.float32)
    x[0] = 0.0
    x[1] *= np.float32(1e-30)                                # squares below binary32
    x[2] *= np.float32(1e30)                                 # squares above it
    x[3] = 3.3e38
    x[4, 1:] = 0.0
    x[5, 3] = np.inf
    x[6, 7] = np.nan
    w = _dev(np.full(k, 0.5, np.float32))
    y = to_np32(w4.w4_rmsnorm(_dev(x), w, 1e-6, out_dtype=F32))
    ref = oracle.rmsnorm_ref(x[:5], np.full(k, 0.5), 1e-6)
    _close(y[:5], ref, 4 * U32 * np.abs(ref) + 2.0 ** -149, "extremes")
    assert np.all(y[0] == 0) and np.isnan(y[5, 3]) and np.isnan(y[6]).all()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    codes, scales = w4.w4_rmsnorm_fp8(_dev(x[:1]), w, 1e-6, status=st)
    assert int(st) == 0 and float(scales) == 1.0 and not codes.any()
    w4.w4_rmsnorm_fp8(_dev(x), w, 1e-6, status=st)
    assert int(st) == 1


def test_rows_past_one_grid_dimension_and_far_offsets():
    # 70000 short rows, and rows whose elements lie past 2^31
    x = _rows(70000, 256, 3, BF)
    w = torch.ones(256, dtype=BF, device=DEV)
    pick = [0, 65534, 65535, 65536, 69999]
    ref = oracle.rmsnorm_ref(to_np32(x[pick]), np.ones(256), 1e-5)
    _close(to_np32(w4.w4_rmsnorm(x, w, 1e-5, out_dtype=F32)[pick]), ref, 4 * U32 * np.abs(ref), "norm")
    y = w4.w4_rmsnorm(x, w, 1e-5, out_dtype=F32)
    codes, scales = w4.w4_rmsnorm_int8(x, w, 1e-5)
    _same_codes(codes[pick], scales[pick], to_np32(y[pick]), "int8", "norm")
    ref = oracle.silu_mul_ref(to_np32(x[pick]))
    got = w4.w4_silu_mul(x, out_dtype=F32)
    _close(to_np32(got[pick]), ref, 8 * U32 * np.abs(ref) + 2.0 ** -126, "gate")
    codes, scales = w4.w4_silu_mul_fp8(x)
    _same_codes(codes[pick], scales[pick], to_np32(got[pick]), "fp8", "gate")
    rows = 270000
    big = torch.zeros(rows, 8192, dtype=BF, device=DEV)
    big[-1] = _rows(1, 8192, 9, BF)[0]
    assert big.numel() > 2 ** 31
    y = w4.w4_rmsnorm(big, torch.ones(8192, dtype=BF, device=DEV), 1e-5)
    ref = oracle.rmsnorm_ref(to_np32(big[-1:]), np.ones(8192), 1e-5)
    _close(to_np32(y[-1:]), ref, (UB + 8 * U32) * np.abs(ref), "last row")
    assert not bool(y[:-1].any())
    del y
    g = w4.w4_silu_mul(big)
    ref = oracle.silu_mul_ref(to_np32(big[-1:]))
    _close(to_np32(g[-1:]), ref, (UB + 16 * U32) * np.abs(ref) + 2.0 ** -126, "last gate row")


@pytest.mark.parametrize("rows,f", NORM_SHAPES)
@pytest.mark.parametrize("xt", [BF, F32])
def test_silu_mul(rows, f, xt):
    _say(f"silu_mul {rows}x{f} {xt}")
    x = _rows(rows, 2 * f, 7 * f + rows, xt)
    ref = oracle.silu_mul_ref(to_np32(x))
    y = w4.w4_silu_mul(x, out_dtype=F32)
    _close(to_np32(y), ref, 8 * U32 * np.abs(ref) + 2.0 ** -126, "f32")
    assert torch.equal(w4.w4_silu_mul(x), y.to(BF))
    for kind, call in (("fp8", w4.w4_silu_mul_fp8), ("int8", w4.w4_silu_mul_int8)):
        codes, scales = call(x)
        _same_codes(codes, scales, to_np32(y), kind, kind)


def test_silu_mul_extremes():
    g = np.array([0.0, -0.0, 1.0, -1.0, 80.0, -80.0, -87.0, -100.0, -3e38, 3e38, 1e-30, -1e-30, 88.8, -88.8, 5.0, np.inf], np.float32)
    x = np.ones((1, 256), np.float32)
    x[0, :16] = g
    y = to_np32(w4.w4_silu_mul(_dev(x), out_dtype=F32))[0]
    ref = oracle.silu_mul_ref(x)[0]
    _close(y[:15], ref[:15], 8 * U32 * np.abs(ref[:15]) + 2.0 ** -126, "extremes")
    assert y[15] == np.inf
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    w4.w4_silu_mul_int8(_dev(x), status=st)
    assert int(st) == 1


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("top", [1.0, 0.37, 2.0 ** -110, 3.0e30])
def test_codes_at_and_next_to_rounding_boundaries(kind, top):
    # silu(64) is 64 in binary32, so y = 64 * u takes any value: quotients at the midpoints between
    # neighbouring codes (exact ties where the scale is a power of two) and up to 40 binary32 ulps
    # around them, zeros of either sign and values that round to zero
    grid = oracle.E4M3_VALUES[:0x7F] if kind == "fp8" else np.arange(128.0)
    most = grid[-1]
    mids = (grid[:-1] + grid[1:]) / 2
    base = np.concatenate([mids, grid])
    near = [base.astype(np.float32)]
    for n in (1, 2, 3, 7, 20, 40):
        near += [(base * (1 + n * 2.0 ** -23)).astype(np.float32), (base * (1 - n * 2.0 ** -24)).astype(np.float32)]
    v = np.concatenate(near)
    v = np.concatenate([v, -v, [0.0, -0.0, 1e-6, -1e-6, 1e-12, -1e-12, 1e-30, -1e-30, most]]).astype(np.float32)
    v = np.minimum(np.maximum(v, -most), most).astype(np.float64) * top
    k = -(-len(v) // 128) * 128
    u = np.zeros((1, k), np.float32)
    u[0, : len(v)] = v / 64
    x = np.concatenate([np.full((1, k), 64.0, np.float32), u], 1)
    y = w4.w4_silu_mul(_dev(x), out_dtype=F32)
    assert np.array_equal(to_np32(y), u * np.float32(64))
    codes, scales = (w4.w4_silu_mul_fp8 if kind == "fp8" else w4.w4_silu_mul_int8)(_dev(x))
    _same_codes(codes, scales, to_np32(y), kind, f"{kind} {top}")


# --------------------------------------------------------------------------
# Rotary positions into the cache
# --------------------------------------------------------------------------

ROPE = [  # tokens, heads, kv, d, rot, interleaved, page, fp8, x dtype, scaling
    (1, 1, 1, 64, 16, False, 16, False, BF, "none"),
    (5, 4, 4, 64, 64, True, 32, True, F32, "linear"),
    (17, 8, 2, 128, 128, False, 16, False, F32, "bands"),
    (33, 64, 8, 128, 128, False, 64, True, BF, "ramp"),
    (9, 6, 2, 128, 80, True, 128, False, BF, "ramp"),
    (9, 5, 1, 128, 96, False, 256, True, F32, "bands"),
    (300, 12, 3, 64, 48, False, 16, False, BF, "none"),
]


@pytest.mark.parametrize("case", ROPE)
def test_rope_cache(case):
    T, heads, kv, d, rot, inter, page, fp8, xt, scaling = case
    _say(f"rope {case}")
    rng = np.random.default_rng(T + rot)
    spec = w4.W4Rope.make(rot, 500000.0, inter, scaling, 1.0 if scaling == "none" else 8.0, 1.0, 32.0 if scaling == "ramp" else 4.0, 8192)
    freqs, amp = w4.w4_rope_frequencies(spec, DEV)
    pages = T // page + 3
    cache = w4.W4KVCache.empty(pages, page, kv, d, fp8=fp8, device=DEV)
    mark = 0x5A if fp8 else -3.0
    for t in (cache.k, cache.v):
        t.fill_(mark)
    x = _rows(T, (heads + 2 * kv) * d, T, xt)
    pos = rng.integers(0, 2_000_000, T).astype(np.int32)
    pos[0] = 0
    if T > 4:
        pos[3] = 2 ** 31 - 1
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    pad = np.zeros(T, bool)
    if T > 2:
        pad[1::4] = True
        slots[pad] = -1
    q0 = torch.full((T, heads, d), 7.0, dtype=BF, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = w4.w4_rope_cache(x, cache, _dev(pos), _dev(slots), spec, freqs, q=q0, status=st)
    assert int(st) == 0
    x3 = to_np32(x).reshape(T, heads + 2 * kv, d)
    ref = oracle.rope_ref(x3[:, : heads + kv], pos, freqs.cpu().numpy(), amp, inter)
    size = oracle.rope_ref(np.abs(x3[:, : heads + kv]), np.zeros(T), np.zeros(rot // 2), amp, inter)   # amplitude * |x|
    half = rot // 2
    i0 = 2 * np.arange(half) if inter else np.arange(half)
    i1 = i0 + 1 if inter else i0 + half
    both = np.zeros_like(size)
    both[..., i0] = both[..., i1] = size[..., i0] + size[..., i1]
    tol = (2 * np.pi * 2.0 ** -26 + 2.0 ** -23 + 4 * U32) * both
    real = ~pad
    got_q = to_np32(q)
    _close(got_q[real], ref[real][:, :heads], tol[real][:, :heads] + UB * (np.abs(ref) + tol)[real][:, :heads], "q")
    assert np.all(got_q[pad] == 7.0)
    kref, ktol, vref = ref[real][:, heads:], tol[real][:, heads:], x3[real][:, heads + kv:]
    at = slots[real]

    def rows_of(t):
        return t.cpu()[at // page, :, at % page]

    if not fp8:
        _close(rows_of(cache.k).float().numpy(), kref, ktol + UB * (np.abs(kref) + ktol), "k")
        assert np.array_equal(rows_of(cache.v).float().numpy(), oracle.bf16_round(vref))
    else:
        rc, rs = oracle.quantize_rows_fp8_ref(vref.reshape(-1, d).astype(np.float32))
        assert np.array_equal(rows_of(cache.v).numpy().reshape(-1, d), rc)
        assert np.array_equal(rows_of(cache.v_scales).numpy().reshape(-1), rs)
        ks = rows_of(cache.k_scales).numpy().astype(np.float64)
        kc = oracle.E4M3_VALUES[rows_of(cache.k).numpy()]
        big = np.abs(kref).max(-1) / 448
        assert np.all(np.abs(ks - big) <= big * U32 + ktol.max(-1) / 448)
        # half a step of the code (2^-4, or 2^-10 below the normal range) on top of the binary32 value
        _close(kc * ks[..., None], kref, ktol * (1 + 2 ** -4) + 2.0 ** -4 * np.abs(kref) * (1 + 4 * U32) + 2.0 ** -10 * ks[..., None] + U32 * np.abs(kref), "k")
    untouched = np.ones(pages * page, bool)
    untouched[at] = False
    for t in (cache.k, cache.v):
        flat = t.transpose(1, 2).reshape(pages * page, -1).cpu()
        assert bool((flat[torch.from_numpy(untouched)] == mark).all())


def test_rope_cache_slots_past_the_cache():
    cache = w4.W4KVCache.empty(2, 16, 1, 64, device=DEV)
    spec = w4.W4Rope.make(64)
    freqs, _ = w4.w4_rope_frequencies(spec, DEV)
    x = _rows(4, 3 * 64, 5, BF)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots = torch.tensor([32, 3, 2 ** 62, -(2 ** 62)], device=DEV)
    q = torch.full((4, 1, 64), 7.0, dtype=BF, device=DEV)
    w4.w4_rope_cache(x, cache, torch.zeros(4, dtype=torch.int32, device=DEV), slots, spec, freqs, q=q, status=st)
    assert int(st) == 8
    assert bool((q[[0, 2, 3]] == 7.0).all()) and not bool((q[1] == 7.0).any())
    assert torch.equal(cache.v[0, 0, 3], x[1, 128:]) and int((cache.v != 0).any(-1).sum()) == 1


def test_rope_cache_nonfinite_row_sets_status():
    cache = w4.W4KVCache.empty(1, 16, 1, 64, fp8=True, device=DEV)
    spec = w4.W4Rope.make(64)
    freqs, _ = w4.w4_rope_frequencies(spec, DEV)
    x = _rows(1, 3 * 64, 5, BF)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    w4.w4_rope_cache(x, cache, zero, zero.long(), spec, freqs, status=st)
    assert int(st) == 0
    x[0, 130] = float("inf")
    w4.w4_rope_cache(x, cache, zero, zero.long(), spec, freqs, status=st)
    assert int(st) == 1


# --------------------------------------------------------------------------
# Block tables
# --------------------------------------------------------------------------

TABLES = [  # B, most new, most cached, page, tokens beyond the sum, pages short, table short, negative
    (1, 1, 0, 16, 0, 0, False, False), (1, 1, 16, 16, 0, 0, False, False), (64, 1, 500, 16, 3, 0, False, False),
    (5, 100, 70, 16, 0, 0, False, False), (300, 9, 200, 32, 10, 0, False, False), (1025, 3, 60, 16, 7, 0, False, False),
    (4096, 5, 40, 16, 1, 0, False, False), (40, 600, 300, 64, 100, 0, False, False), (20, 30, 90, 16, 0, 25, False, False),
    (20, 30, 90, 16, -100, 0, False, False), (20, 30, 90, 16, 5, 0, True, False), (50, 30, 90, 16, 5, 10, True, True),
    (30, 900, 64, 16, -3000, 40, False, True),
]


@pytest.mark.parametrize("case", TABLES)
@pytest.mark.parametrize("in_place", [False, True])
def test_block_tables(case, in_place):
    B, most, old, page, extra, short, narrow, negative = case
    _say(f"tables {case}")
    rng = np.random.default_rng(B * 31 + most)
    new = rng.integers(0, most + 1, B).astype(np.int32)
    new[0] = most
    lens = rng.integers(0, old + 1, B).astype(np.int32)
    if negative:
        new[3], lens[5] = -4, -7
    have, want = -(-np.maximum(lens, 0) // page), -(-(np.maximum(lens, 0) + np.maximum(new, 0)) // page)
    wide = max(1, int(want.max()) - (2 if narrow else 0))
    taken = int((want - have).sum())
    pool = int(have.sum()) + taken + 9
    order = rng.permutation(pool).astype(np.int32)
    table = np.full((B, wide), -1, np.int32)
    used = 0
    for b in range(B):
        n = min(int(have[b]), wide)
        table[b, :n] = order[used: used + n]
        used += n
    free = order[used:]
    count = max(0, taken + 4 - short)
    free, tokens = np.ascontiguousarray(free), max(1, int(np.maximum(new, 0).sum()) + extra)
    cu, pos, slots, lens_ref, left, table_ref, status = oracle.block_tables_ref(new, lens, free, count, table, page, tokens)
    d_lens, d_count, d_table = _dev(lens), _dev(np.array([count], np.int32)), _dev(table)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = {} if in_place else dict(lens_out=torch.full_like(d_lens, -9), free_count_out=torch.full_like(d_count, -9))
    got = w4.w4_block_tables(_dev(new), d_lens, _dev(free), d_count, d_table, page, tokens=tokens, status=st, **kw)
    assert got[0].cpu().tolist() == cu
    assert got[1].cpu().tolist() == pos
    assert got[2].cpu().tolist() == slots
    assert kw.get("lens_out", d_lens).cpu().tolist() == lens_ref
    assert int(kw.get("free_count_out", d_count)) == left
    assert d_table.cpu().tolist() == table_ref
    assert int(st) == status


def test_block_tables_step_by_step():
    # decode steps in place, captured once and replayed: lengths and list move on as in eager steps
    B, page, steps = 6, 16, 40
    dev = [torch.device(DEV)]

    def state():
        return dict(lens=torch.tensor([0, 1, 15, 16, 30, 31], dtype=torch.int32, device=DEV),
                    free=torch.arange(100, dtype=torch.int32, device=DEV), count=torch.full((1,), 60, dtype=torch.int32, device=DEV),
                    table=torch.cat([torch.full((B, 1), 60, dtype=torch.int32, device=DEV) + torch.arange(B, dtype=torch.int32, device=DEV)[:, None],
                                     torch.full((B, 5), -1, dtype=torch.int32, device=DEV)], 1).contiguous(),
                    new=torch.ones(B, dtype=torch.int32, device=DEV))

    a, b = state(), state()
    for s in (a, b):
        s["table"][4, 1], s["table"][5, 1] = 70, 71
        s["out"] = dict(cu_q=torch.empty(B + 1, dtype=torch.int32, device=DEV), positions=torch.empty(B, dtype=torch.int32, device=DEV),
                        slots=torch.empty(B, dtype=torch.int64, device=DEV))

    def step(s):
        w4.w4_block_tables(s["new"], s["lens"], s["free"], s["count"], s["table"], page, **s["out"])

    step(a)
    step(b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(b)
    del dev
    for i in range(steps):
        step(a)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n in ("lens", "count", "table"):
            assert torch.equal(a[n], b[n]), (i, n)
        assert torch.equal(a["out"]["slots"], b["out"]["slots"])
    assert a["lens"].cpu().tolist() == [41, 42, 56, 57, 71, 72]


# --------------------------------------------------------------------------
# Attention
# --------------------------------------------------------------------------

class Batch:
    """Requests over a shuffled paged cache whose unused rows hold NaN."""

    def __init__(self, new, cached, heads, kv, d, page, fp8, seed=0, pad=0, wide=0, qscale=1.0):
        rng = np.random.default_rng(seed)
        self.new, self.ctx = list(new), [n + c for n, c in zip(new, cached)]
        self.heads, self.kv, self.d, self.page, self.fp8 = heads, kv, d, page, fp8
        need = [-(-c // page) for c in self.ctx]
        pages = sum(need) + 2
        order = rng.permutation(pages)
        width = max(max(need), 1) + wide
        self.table = np.full((len(need), width), -1, np.int32)
        used = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[used: used + n]
            used += n
        self.keys, self.values = [], []
        shape = (pages, kv, page, d)
        if fp8:
            raw = {n: np.full(shape, 0x7F, np.uint8) for n in "kv"}
            sc = {n: np.full(shape[:3], np.nan, np.float32) for n in "kv"}
        else:
            raw = {n: np.full(shape, np.nan, np.float32) for n in "kv"}
        for b, c in enumerate(self.ctx):
            j = np.arange(c)
            pg, at = self.table[b, j // page], j % page
            for n, store in (("k", self.keys), ("v", self.values)):
                x = oracle.bf16_round(rng.standard_normal((c, kv, d)).astype(np.float32))
                if fp8:
                    codes, s = oracle.quantize_rows_fp8_ref(x.reshape(-1, d)) if c else (np.zeros((0, d), np.uint8), np.zeros(0, np.float32))
                    raw[n][pg, :, at] = codes.reshape(c, kv, d)
                    sc[n][pg, :, at] = s.reshape(c, kv)
                    x = oracle.E4M3_VALUES[codes].reshape(c, kv, d) * s.reshape(c, kv, 1).astype(np.float64)
                else:
                    raw[n][pg, :, at] = x
                store.append(x.transpose(1, 0, 2))
        self.cache = (w4.W4KVCache(_dev(raw["k"]), _dev(raw["v"]), _dev(sc["k"]), _dev(sc["v"])) if fp8
                      else w4.W4KVCache(_dev(raw["k"], BF), _dev(raw["v"], BF)))
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.q = oracle.bf16_round((qscale * rng.standard_normal((int(self.cu[-1]) + pad, heads, d))).astype(np.float32))
        self.d_q, self.d_table, self.d_cu = _dev(self.q, BF), _dev(self.table), _dev(self.cu)
        self.d_lens = _dev(np.array(self.ctx, np.int32))
        self.scale = d ** -0.5

    def run(self, window=0, **kw):
        o = torch.full(self.q.shape, 7.0, dtype=BF, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        need = w4.w4_paged_attention_workspace_bytes(self.q.shape[0], self.heads, self.cache, len(self.new), self.table.shape[1])
        ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device=DEV)   # NaN in every part
        args = dict(o=o, workspace=ws, status=st)
        args.update(kw)
        got = w4.w4_paged_attention(self.d_q, self.cache, self.d_table, self.d_cu, self.d_lens, self.scale, window=window, **args)
        self.status = int(st)
        return got

    def check(self, got, window=0, what="", status=0):
        assert self.status == status, what
        got = to_np32(got)
        for b, n in enumerate(self.new):
            s = slice(int(self.cu[b]), int(self.cu[b]) + n)
            if n == 0:
                continue
            q = self.q[s]
            ref, weight = oracle.attention_ref(q, self.keys[b], self.values[b], self.ctx[b], self.scale, window)
            size = self.scale * np.abs(q).sum(-1).max() * (np.abs(self.keys[b]).max() if self.ctx[b] else 0)
            score = (self.d + 2) * U32 * size + size * 1.5 * U32
            tol = (UB + 2 * (score + (4 + self.ctx[b] / 8) * U32)) * weight + UB * np.abs(ref) + 2.0 ** -100
            _close(got[s], ref, tol, f"{what} request {b}")
        assert np.all(got[int(self.cu[-1]):] == 7.0), f"{what}: rows behind the last request"


ATTEND = [  # new, cached, heads, kv, d, page, fp8, window
    ([1], [0], 1, 1, 64, 16, False, 0),
    ([1], [0], 4, 1, 128, 16, True, 0),
    ([1], [15], 8, 8, 128, 16, False, 0),
    ([1], [16], 8, 8, 64, 16, True, 0),
    ([1], [31], 32, 1, 64, 32, False, 0),
    ([1], [63], 40, 1, 128, 16, False, 0),                    # more heads than a tile has rows
    ([1], [1000], 32, 32, 128, 16, False, 0),
    ([1], [4095], 16, 2, 128, 64, False, 0),
    ([1], [20001], 8, 1, 128, 64, True, 0),
    ([1], [9000], 3, 1, 64, 128, False, 0),
    ([1] * 7, [0, 1, 30, 31, 32, 500, 3001], 12, 4, 128, 16, False, 0),
    ([1] * 5, [900, 1, 64, 65, 129], 10, 2, 64, 256, True, 0),
    ([3, 0, 4, 1], [5, 9, 60, 700], 8, 1, 128, 16, False, 0),  # 24, 0, 32 and 8 rows
    ([5, 1, 0, 40], [0, 100, 3, 77], 8, 1, 128, 32, True, 0),  # both kernels
    ([33], [0], 4, 4, 64, 16, False, 0),
    ([64], [64], 2, 2, 128, 16, False, 0),
    ([300], [0], 4, 4, 128, 32, False, 0),
    ([257], [1000], 6, 2, 64, 64, True, 0),
    ([130, 1, 70, 1, 1], [500, 2000, 0, 63, 64], 16, 2, 128, 16, False, 0),
    ([600], [5000], 8, 1, 128, 128, False, 0),                # few tiles over many keys: split
    ([100], [3000], 8, 8, 128, 64, True, 0),
    ([1] * 4, [200, 5, 700, 64], 8, 2, 128, 16, False, 64),
    ([1] * 2, [5000, 9000], 8, 2, 64, 16, True, 1),
    ([1] * 2, [5000, 9000], 8, 2, 128, 16, False, 3000),
    ([200, 3], [100, 400], 4, 2, 128, 16, False, 33),
    ([300], [700], 2, 1, 64, 64, False, 500),
    ([64, 64], [0, 64], 5, 5, 128, 16, True, 1),
    ([6, 0, 0, 0, 0, 0, 3, 0, 0], [100, 5, 6, 7, 8, 9, 50, 1, 2], 8, 1, 128, 16, False, 0),  # as many tokens as requests, not one each
    ([1] * 65, [(7 * i) % 90 for i in range(65)], 4, 2, 64, 16, False, 0),                    # more requests than lanes
    ([i % 3 for i in range(200)], [(11 * i) % 60 for i in range(200)], 4, 1, 64, 16, True, 0),
    ([40 * (i % 50 == 49) + (i % 2) for i in range(150)], [(5 * i) % 40 for i in range(150)], 8, 2, 64, 16, False, 0),
    ([1, 5], [5000, 4200], 4, 2, 64, 4096, False, 0),
    ([1] * 3, [40, 3000, 1200], 24, 1, 128, 16, False, 0),    # more heads of a kv head than a tile has rows
    ([1] * 2, [700, 9000], 40, 1, 64, 32, True, 100),
    ([1, 3, 40], [6000, 5000, 9], 16, 2, 128, 16, False, 0),  # 8, 24 and 320 rows, the few split over the keys
    ([2, 1, 50], [4000, 3, 9], 17, 1, 64, 16, True, 0),       # 34, 17 and 850 rows
    ([3], [700], 8, 1, 128, 16, False, 0),                    # few rows in all: 24, 16 and 32
    ([1] * 9, [7000, 1, 300, 0, 31, 5000, 63, 64, 90], 32, 1, 128, 16, False, 0),   # 32 rows a tile
    ([1] * 6, [3000, 9, 4000, 77, 512, 513], 50, 2, 64, 16, True, 0),
    ([2, 1, 0, 1], [2000, 700, 60, 31], 20, 1, 128, 16, True, 50),
    ([1] * 4, [6000, 200, 0, 900], 33, 1, 128, 64, False, 0),
    ([0, 1, 0], [5, 70000, 3], 20, 1, 64, 64, False, 0),      # one token of three requests
    ([6, 1, 8, 30, 5], [3000, 900, 40, 7, 1000], 16, 2, 128, 16, False, 0),   # 48, 8, 64, 240 and 40 rows
    ([9, 0, 1, 60, 7], [2500, 9, 4000, 300, 31], 7, 1, 64, 32, True, 200),    # 63, 0, 7, 420 and 49 rows
    ([2, 0, 2], [30, 4, 2000], 8, 2, 64, 16, True, 0),
    ([31, 1], [3, 5000], 4, 4, 128, 32, False, 40),
    ([300, 1300], [4500, 100], 32, 8, 64, 64, False, 0),      # split and unsplit tiles in one call
    ([300, 1, 1300], [4500, 900, 100], 32, 8, 64, 64, False, 700),
]


@pytest.mark.parametrize("case", ATTEND)
def test_attention(case):
    new, cached, heads, kv, d, page, fp8, window = case
    _say(f"attention {case}")
    b = Batch(new, cached, heads, kv, d, page, fp8, seed=len(new) + heads, pad=3, wide=2)
    b.check(b.run(window), window, str(case))


@pytest.mark.parametrize("d,fp8", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("new,cached", [([1, 1], [2000, 999]), ([150], [900])])
def test_attention_counts_every_key_once(d, fp8, new, cached):
    # scores all 0: the output is the share of the visible keys j with j % d == column
    b = Batch(new, cached, 4, 2, d, 16, fp8, seed=3)
    b.d_q.zero_()
    for i, c in enumerate(b.ctx):
        j = np.arange(c)
        v = np.zeros((c, 2, d), np.float32)
        v[j, :, j % d] = 1.0
        pg, at = torch.from_numpy(b.table[i, j // 16].astype(np.int64)).to(DEV), torch.from_numpy(j % 16).to(DEV)
        if fp8:
            b.cache.v[pg, :, at] = _dev((v * 0x38).astype(np.uint8))     # 0x38: one in E4M3
            b.cache.v_scales[pg, :, at] = 1.0
        else:
            b.cache.v[pg, :, at] = _dev(v, BF)
    got = to_np32(b.run())
    for i, n in enumerate(new):
        for t in range(n):
            seen = b.ctx[i] - n + t + 1
            ref = np.array([len(range(c, seen, d)) for c in range(d)]) / seen
            row = got[int(b.cu[i]) + t]
            assert np.all(np.abs(row - ref) <= (UB + 4 * U32) * ref), (i, t)


def test_attention_large_scores_and_slack():
    # scores of hundreds that grow along the context: every step raises the maximum
    for new, cached in (([1], [3000]), ([80], [800])):
        b = Batch(new, cached, 8, 2, 128, 16, False, seed=9, qscale=40.0)
        b.check(b.run(), 0, "large scores")
        k = b.cache.k
        up = torch.arange(b.ctx[0], device=DEV) / 50.0
        j = np.arange(b.ctx[0])
        pg, at = torch.from_numpy(b.table[0, j // 16].astype(np.int64)).to(DEV), torch.from_numpy(j % 16).to(DEV)
        k[pg, :, at] = (up[:, None, None] / 11.3 * torch.ones(1, 2, 128, device=DEV)).to(BF)
        b.d_q.fill_(1.0)
        b.q[:] = 1.0
        b.keys[0] = np.broadcast_to(to_np32(k[pg, :, at]).transpose(1, 0, 2), b.keys[0].shape)
        b.check(b.run(), 0, "rising scores")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,cached,window", [([40], [100], 0), ([3, 50, 1], [10, 0, 800], 0), ([300], [900], 64), ([1, 1], [3000, 70], 50),
                                               ([2, 1], [1500, 70], 0)])
def test_attention_keeps_masked_values_out(fp8, new, cached, window):
    # an infinity or NaN at a key reaches the rows that see the key and no other
    b = Batch(new, cached, 8, 2, 128, 16, fp8, seed=21)
    clean = to_np32(b.run(window))
    b.check(b.run(window), window, "clean")
    for which, value in (("v", float("nan")), ("v", float("inf")), ("k", float("nan"))):
        c = Batch(new, cached, 8, 2, 128, 16, fp8, seed=21)
        hit = [(i, max(0, n_c - 1 - (n > 2) * 7)) for i, (n, n_c) in enumerate(zip(new, c.ctx))]
        for i, j in hit:
            row = getattr(c.cache, which)[int(c.table[i, j // 16]), :, j % 16]
            if fp8:
                row[:, 5] = 0x7F
                if value == float("inf"):
                    getattr(c.cache, which + "_scales")[int(c.table[i, j // 16]), :, j % 16] = float("inf")
            else:
                row[:, 5] = value
        got = to_np32(c.run(window))
        for (i, j), n in zip(hit, new):
            for t in range(n):
                pos = c.ctx[i] - n + t
                row, was = got[int(c.cu[i]) + t], clean[int(c.cu[i]) + t]
                if j <= pos and (not window or j > pos - window):
                    assert not np.isfinite(row[:, 5]).any(), (which, value, i, t)
                    if which == "k":
                        assert np.isnan(row).all()
                else:
                    assert np.all(np.abs(row - was) <= 4 * UB * np.abs(was) + 0.02), (which, value, i, t)


def test_attention_empty_rows_and_bad_lengths():
    # lens below the new tokens: the first rows see nothing; 0 and negative; longer than the table
    b = Batch([4, 2, 3, 1], [60, 10, 20, 30], 8, 2, 64, 16, False, seed=4, pad=2)
    ctx = [2, 0, -5, 31]
    b.d_lens = _dev(np.array(ctx, np.int32))
    got = to_np32(b.run())
    assert b.status == 0
    assert np.all(got[:2] == 0) and np.all(got[4:9] == 0) and np.all(got[10:] == 7.0)
    for rows, i, c in ((slice(2, 4), 0, 2), (slice(9, 10), 3, 31)):
        ref, w = oracle.attention_ref(b.q[rows], b.keys[i][:, :c], b.values[i][:, :c], c, b.scale)
        _close(got[rows], ref, (UB + 1e-4) * w + UB * np.abs(ref), "short")
    b.d_lens = _dev(np.array([2 ** 31 - 1] * 4, np.int32))     # clamped to the table: entries of -1 are reported
    b.run()
    assert b.status == 8
    b.d_cu = _dev(np.array([0, -7, 2 ** 31 - 1, 5, 3], np.int32))
    b.run()


def test_attention_bad_pages_read_as_zeros():
    for new, cached in (([1], [199]), ([90], [110])):
        b = Batch(new, cached, 4, 2, 128, 16, False, seed=6)
        keep = b.table.copy()
        for entry, value in ((2, -1), (5, b.cache.pages), (7, 2 ** 31 - 1), (9, -(2 ** 31))):
            b.table[0, entry] = value
            for x in (b.keys[0], b.values[0]):
                x[:, entry * 16: entry * 16 + 16] = 0.0
        b.d_table = _dev(b.table)
        b.check(b.run(), 0, "bad pages", status=8)
        b.d_table = _dev(keep)


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_of_32_row_tiles_redone(fp8):
    # 24 rows of one request beside a chunk: a NaN that only its later tokens see, then pages that are not there
    new, cached = [12, 40], [900, 10]
    b = Batch(new, cached, 4, 2, 128, 16, fp8, seed=23)
    clean = to_np32(b.run())
    b.check(b.run(), 0, "clean")
    c = Batch(new, cached, 4, 2, 128, 16, fp8, seed=23)
    j = c.ctx[0] - 8
    c.cache.v[int(c.table[0, j // 16]), :, j % 16, 5] = 0x7F if fp8 else float("nan")
    got = to_np32(c.run())
    assert np.all(np.abs(got[:4] - clean[:4]) <= 4 * UB * np.abs(clean[:4]) + 0.02)
    assert np.isnan(got[4:12, :, 5]).all() and np.isfinite(got[4:12, :, :5]).all()
    assert np.array_equal(got[12:], clean[12:])
    for entry, value in ((3, -1), (40, b.cache.pages)):
        b.table[0, entry] = value
        for x in (b.keys[0], b.values[0]):
            x[:, entry * 16: entry * 16 + 16] = 0.0
    b.d_table = _dev(b.table)
    b.check(b.run(), 0, "bad pages", status=8)


@pytest.mark.parametrize("new,cached", [([1] * 3, [3000, 40, 900]), ([70, 1, 4], [2000, 300, 5])])
def test_attention_graph_and_streams(new, cached):
    b = Batch(new, cached, 16, 2, 128, 16, False, seed=8)
    ref = b.run()
    need = w4.w4_paged_attention_workspace_bytes(b.q.shape[0], 16, b.cache, len(new), b.table.shape[1])
    bufs = [dict(o=torch.zeros_like(ref), workspace=torch.empty(max(need, 1), dtype=torch.uint8, device=DEV), status=None) for _ in range(2)]
    for _ in range(3):                                        # the same call twice is the same to the bit
        assert torch.equal(b.run(), ref)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.w4_paged_attention(b.d_q, b.cache, b.d_table, b.d_cu, b.d_lens, b.scale, **{k: v for k, v in bufs[0].items()})
    for _ in range(3):
        bufs[0]["o"].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs[0]["o"], ref)
        assert torch.equal(b.run(), ref)
    # shorter contexts in the same graph
    lens = b.d_lens.clone()
    b.d_lens.sub_(torch.tensor([7] + [0] * (len(new) - 1), dtype=torch.int32, device=DEV))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(bufs[0]["o"], b.run())
    b.d_lens.copy_(lens)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, buf in zip(side, bufs):                            # two calls at once, with a workspace each
        with torch.cuda.stream(s):
            for _ in range(5):
                w4.w4_paged_attention(b.d_q, b.cache, b.d_table, b.d_cu, b.d_lens, b.scale, **{k: v for k, v in buf.items()})
    torch.cuda.synchronize()
    assert torch.equal(bufs[0]["o"], ref) and torch.equal(bufs[1]["o"], ref)


def test_attention_of_most_requests():
    # 4096 requests, a few of them with tokens or keys: scores 0, so each row is the mean of its values
    B, d = 4096, 64
    rng = np.random.default_rng(2)
    new = (rng.random(B) < 0.2).astype(np.int32)
    new[-1], new[0], new[63], new[64], new[4032] = 2, 1, 0, 1, 3
    ctx = np.where(new > 0, new + rng.integers(0, 14, B), 0).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    v = torch.arange(B * 16, device=DEV, dtype=F32).remainder(97).view(B, 1, 16, 1).expand(B, 1, 16, d).contiguous().to(BF)
    cache = w4.W4KVCache(torch.zeros_like(v), v)
    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None].contiguous()
    o = w4.w4_paged_attention(torch.zeros(T, 2, d, dtype=BF, device=DEV), cache, table, _dev(cu), _dev(ctx), 1.0)
    got, vals = to_np32(o), to_np32(v)[:, 0, :, 0].astype(np.float64)
    for b in np.nonzero(new)[0]:
        for t in range(new[b]):
            ref = vals[b, : ctx[b] - new[b] + t + 1].mean()
            assert np.all(np.abs(got[cu[b] + t] - ref) <= (UB + 2.0 ** -14) * ref), (b, t)


def test_attention_of_most_tiles():
    # as many requests and kv heads as there may be: more workgroups than one grid dimension holds
    B, kv, d, pages = 4096, 1024, 64, 8
    new = np.ones(B, np.int32)
    new[7] = 2
    ctx = (new + np.arange(B) % 13).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    v = torch.arange(pages * 16, device=DEV, dtype=F32).remainder(97).view(pages, 1, 16, 1).expand(pages, kv, 16, d).contiguous().to(BF)
    cache = w4.W4KVCache(torch.zeros_like(v), v)
    table = (torch.arange(B, dtype=torch.int32, device=DEV) % pages)[:, None].contiguous()
    _say("attention of 4096 requests and 1024 kv heads")
    o = w4.w4_paged_attention(torch.zeros(T, kv, d, dtype=BF, device=DEV), cache, table, _dev(cu), _dev(ctx), 1.0)
    vals = to_np32(v)[:, 0, :, 0].astype(np.float64)
    ref = np.concatenate([[vals[b % pages, : ctx[b] - new[b] + t + 1].mean() for t in range(new[b])] for b in range(B)])
    ref = torch.from_numpy(ref).to(DEV, F32).view(T, 1, 1)     # off by 2^-24 of itself, inside the 2^-14 below
    assert bool(((o.float() - ref).abs() <= (UB + 2.0 ** -14) * ref).all())


def test_attention_far_offsets():
    # a cache past 2^32 bytes: pages at its end are reached with 64-bit offsets
    pages, page, kv, d = 300_000, 16, 8, 128
    k = torch.zeros(pages, kv, page, d, dtype=BF, device=DEV)
    v = torch.zeros(pages, kv, page, d, dtype=BF, device=DEV)
    assert k.numel() * 2 > 2 ** 33
    cache = w4.W4KVCache(k, v)
    table = torch.tensor([[pages - 1, 0, pages - 2, 7]], dtype=torch.int32, device=DEV)
    for i, p in enumerate(table[0].tolist()):
        v[p] = i + 1.0
    q = torch.zeros(1, 8, d, dtype=BF, device=DEV)
    o = w4.w4_paged_attention(q, cache, table, torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                              torch.tensor([64], dtype=torch.int32, device=DEV), 1.0)
    assert bool((o == 2.5).all())


# --------------------------------------------------------------------------
# Refusals of the Python layer that need device tensors
# --------------------------------------------------------------------------

def test_python_layer_refusals():
    x = torch.zeros(4, 256, dtype=BF, device=DEV)
    w = torch.ones(256, dtype=BF, device=DEV)
    with pytest.raises(ValueError):
        w4.w4_rmsnorm(x[:, ::2], w[::2], 1e-5)
    with pytest.raises(ValueError):
        w4.w4_rmsnorm(x, w[:128], 1e-5)
    with pytest.raises(ValueError):
        w4.w4_rmsnorm(x, w, 1e-5, residual_out=x)
    with pytest.raises(TypeError):
        w4.w4_rmsnorm(x.half(), w, 1e-5)
    with pytest.raises(TypeError):
        w4.w4_rmsnorm(x, w, 1e-5, residual=x.clone(), residual_out=x.float())
    with pytest.raises(w4.W4Error) as e:
        w4.w4_rmsnorm(x, w, 0.0)
    assert e.value.status == 10
    with pytest.raises(ValueError):
        w4.w4_rmsnorm(x, w.cpu(), 1e-5)
    with pytest.raises(TypeError):
        w4.w4_silu_mul_fp8(x, codes=torch.zeros(4, 128, dtype=torch.int8, device=DEV))
    with pytest.raises(w4.W4Error):
        w4.w4_silu_mul(torch.zeros(4, 300, dtype=BF, device=DEV))
    with pytest.raises(ValueError):
        w4.w4_silu_mul(torch.zeros(4, 257, dtype=BF, device=DEV))
    c = w4.W4KVCache.empty(2, 16, 1, 64, device=DEV)
    with pytest.raises(ValueError):
        w4.W4KVCache(c.k, c.v, torch.ones(2, 1, 16, device=DEV))
    with pytest.raises(TypeError):
        w4.W4KVCache(c.k, c.v.float())
    q = torch.zeros(1, 2, 64, dtype=BF, device=DEV)
    i = torch.zeros(1, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        w4.w4_paged_attention(q[:, :, :32], c, i[None], torch.zeros(2, dtype=torch.int32, device=DEV), i, 1.0)
    with pytest.raises(ValueError):
        w4.w4_paged_attention(q, c, i[None], i, i, 1.0)
    with pytest.raises(TypeError):
        w4.w4_paged_attention(q, c, i[None].long(), torch.zeros(2, dtype=torch.int32, device=DEV), i, 1.0)
    with pytest.raises(w4.W4Error) as e:
        w4.w4_paged_attention(q, c, i[None], torch.zeros(2, dtype=torch.int32, device=DEV), i, -1.0)
    assert e.value.status == 10
    big = torch.zeros(1, 4096, dtype=torch.int32, device=DEV)
    with pytest.raises(w4.W4Error) as e:
        w4.w4_paged_attention(q, c, big, torch.zeros(2, dtype=torch.int32, device=DEV), i, 1.0, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 7
