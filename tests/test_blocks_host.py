"""Host-side checks of the INT8 cache and of the attention's other scores (no GPU needed): refusals before any
device work, record sizes, the key ranges that the kernels share with the host, and the oracle's own pins.
No call here passes validation, so no kernel is launched.
"""

import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

import dequant_gemv_w4_amd as w4
import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL = ctypes.c_void_p(None)
OK_ADDR = 0x100000


def f(addr=OK_ADDR):
    return ctypes.c_void_p(addr)


def cache(**kw):
    d = dict(k=OK_ADDR, v=OK_ADDR, k_scales=OK_ADDR, v_scales=OK_ADDR, pages=10, page_size=16, kv_heads=2, head_dim=128, type=3)
    d.update(kw)
    return ctypes.byref(w4._KVCacheStruct(**d))


BAD_CACHES = [(dict(type=2), 5), (dict(type=4), 5), (dict(type=-1), 5), (dict(head_dim=96), 5), (dict(page_size=8), 5),
              (dict(page_size=48), 5), (dict(kv_heads=0), 2), (dict(pages=0), 2), (dict(k=None), 1), (dict(v=None), 1),
              (dict(k_scales=None), 1), (dict(v_scales=None), 1), (dict(k=OK_ADDR + 8), 3), (dict(v_scales=OK_ADDR + 2), 3)]


def test_write_refusals():
    L = w4.lib()

    def call(x=f(), xt=1, T=3, heads=4, c=None, slots=f(), q=f(), st=NULL):
        return L.w4_cache_write(x, xt, T, heads, c or cache(), slots, q, st, NULL)

    for name in ("x", "slots", "q"):
        assert call(**{name: NULL}) == 1, name
    assert L.w4_cache_write(f(), 1, 3, 4, None, f(), f(), NULL, NULL) == 1
    assert call(xt=2) == 4 and call(xt=-1) == 4
    assert call(T=0) == 2 and call(T=(1 << 22) + 1) == 2 and call(heads=3) == 2 and call(heads=1) == 2 and call(heads=-2) == 2
    assert call(T=1 << 22, heads=16) == 2 and call(T=1, heads=65538) == 2
    assert call(T=1 << 22, heads=0, q=NULL, c=cache(kv_heads=16)) == 2
    for kw, status in BAD_CACHES:
        assert call(c=cache(**kw)) == status, kw
    assert call(x=f(OK_ADDR + 8)) == 3 and call(q=f(OK_ADDR + 8)) == 3 and call(slots=f(OK_ADDR + 4)) == 3 and call(st=f(OK_ADDR + 2)) == 3
    r = ctypes.byref(w4.W4Rope.make(64))
    for kw, status in BAD_CACHES:
        assert L.w4_rope_cache(f(), 1, 3, 4, cache(**kw), f(), f(), r, f(), f(), NULL, NULL) == status, kw


def test_read_refusals():
    L = w4.lib()

    def call(c=None, slots=f(), n=3, kv=f(), yt=1, st=NULL):
        return L.w4_cache_read(c or cache(), slots, n, kv, yt, st, NULL)

    assert L.w4_cache_read(None, f(), 3, f(), 1, NULL, NULL) == 1
    assert call(slots=NULL) == 1 and call(kv=NULL) == 1 and call(yt=2) == 4
    assert call(n=0) == 2 and call(n=-1) == 2 and call(n=(1 << 22) + 1) == 2
    for kw, status in BAD_CACHES:
        assert call(c=cache(**kw)) == status, kw
    assert call(slots=f(OK_ADDR + 4)) == 3 and call(kv=f(OK_ADDR + 8)) == 3 and call(st=f(OK_ADDR + 1)) == 3


def scores(**kw):
    d = dict(cap=0.0, reserved=0, slopes=None, first_keys=None, prefix_lens=None)
    d.update(kw)
    return ctypes.byref(w4._ScoresStruct(**d))


def test_scores_refusals():
    L = w4.lib()
    assert ctypes.sizeof(w4._ScoresStruct) == 32

    def call(q=f(), T=3, heads=4, c=None, bt=f(), mp=4, cu=f(), lens=f(), B=2, scale=0.1, window=0, s=None, o=f(), ws=f(), wb=1 << 30, st=NULL):
        return L.w4_paged_attention_scores(q, T, heads, c or cache(), bt, mp, cu, lens, B, scale, window, s or scores(cap=30.0),
                                           o, ws, wb, st, NULL)

    for name in ("q", "bt", "cu", "lens", "o"):
        assert call(**{name: NULL}) == 1, name
    assert L.w4_paged_attention_scores(f(), 3, 4, cache(), f(), 4, f(), f(), 2, 0.1, 0, None, f(), f(), 1 << 30, NULL, NULL) == 1
    assert call(T=0) == 2 and call(heads=3) == 2 and call(B=0) == 2 and call(B=4097) == 2 and call(mp=0) == 2 and call(mp=1 << 27) == 2
    for kw, status in BAD_CACHES:
        assert call(c=cache(**kw)) == status, kw
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=scale) == 10
    assert call(window=-1) == 10
    assert call(s=scores(reserved=1)) == 5
    # the cap: within 2^20 of the scale either way, and scales up to 256 then
    for cap in (-1.0, math.nan, math.inf, -math.inf, 0.1 * 2.0 ** 21, 0.1 * 2.0 ** -21, 1e-30):
        assert call(s=scores(cap=cap)) == 10, cap
    assert call(scale=257.0, s=scores(cap=257.0)) == 10
    for name in ("slopes", "first_keys", "prefix_lens"):
        assert call(s=scores(**{name: OK_ADDR + 2})) == 3, name
    assert call(q=f(OK_ADDR + 8)) == 3 and call(o=f(OK_ADDR + 8)) == 3 and call(ws=f(OK_ADDR + 8)) == 3
    long = dict(T=1, heads=2, B=1, mp=4096)                   # keys split over workgroups: a workspace is needed
    assert call(ws=NULL, wb=0, **long) == 7 and call(wb=16, **long) == 7
    # a workspace size goes by the geometry alone, of either 8-bit type
    for t, c in ((1, cache(type=1)), (3, cache())):
        assert L.w4_paged_attention_workspace_bytes(1, 2, c, 1, 4096) > 0, t


def test_python_layer_rejects_cpu_tensors():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        w4.W4KVCache(torch.zeros(2, 1, 16, 64, dtype=torch.int8), torch.zeros(2, 1, 16, 64, dtype=torch.int8))
    with pytest.raises(ValueError):
        w4.W4Scores(slopes=torch.zeros(4))
    with pytest.raises(TypeError):
        w4.W4Scores(first_keys=[0, 1])


def test_scores_keep_what_they_were_made_with():
    pytest.importorskip("torch")
    r = w4.W4Scores(cap=30.0)
    for name, value in (("cap", 50.0), ("slopes", None), ("first_keys", None), ("prefix_lens", None)):
        with pytest.raises(AttributeError):
            setattr(r, name, value)
    assert r.cap == 30.0 and r._c.cap == 30.0


PROGRAM = r"""
#include <cstdio>
#include <climits>
#include <vector>
#include "w4_paging.h"
using namespace w4;
static uint64_t state = 88172645463325252ull;
static int64_t rnd(int64_t lo, int64_t hi) {
    state ^= state << 13; state ^= state >> 7; state ^= state << 17;
    return lo + (int64_t)(state % (uint64_t)(hi - lo + 1));
}
#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
int main() {
    const int32_t far[] = {INT32_MIN, INT32_MIN + 1, -1, 0, 1, INT32_MAX - 1, INT32_MAX};
    for (int trial = 0; trial < 200000; ++trial) {
        const int32_t ctx = (int32_t)rnd(0, 300), pos = (int32_t)rnd(-40, ctx - 1), window = rnd(0, 1) ? (int32_t)rnd(1, 200) : 0;
        const int32_t first = rnd(0, 4) ? (int32_t)rnd(-20, 320) : far[rnd(0, 6)];
        const int32_t prefix = rnd(0, 4) ? (int32_t)rnd(-20, 320) : far[rnd(0, 6)];
        const KeyRange k = key_range(pos, ctx, window, first, prefix);
        CHECK(k.lo >= 0 && k.hi < ctx);
        for (int64_t j = 0; j < ctx; ++j) {
            const bool seen = (j <= pos || j < prefix) && j >= first && (window == 0 || j >= (int64_t)pos - window + 1);
            CHECK(seen == (j >= k.lo && j <= k.hi));
        }
        // the span that a range is cut into: every key of it in exactly one part, no part ahead of its 16 keys
        if (k.lo > k.hi) continue;
        const int32_t parts = (int32_t)rnd(1, 9), least = 64 * (int32_t)rnd(1, 4);
        const Span s = seen_span(cut_span(k.lo, k.hi + 1, parts, least));
        CHECK(s.parts >= 1 && s.parts <= parts && s.begin % 16 == 0 && s.begin <= k.lo && s.begin + 16 > k.lo && s.end == k.hi + 1);
        CHECK(s.begin + (int64_t)s.parts * s.chunk >= s.end && s.begin + (int64_t)(s.parts - 1) * s.chunk < s.end);
    }
    const Span none = seen_span(cut_span(0, 0, 8, 128));
    CHECK(none.parts == 1 && none.begin == none.end);
    std::puts("ok");
}
"""


def test_key_ranges(tmp_path):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "ranges.cpp", tmp_path / "ranges"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I",
                    os.path.join(ROOT, "dequant_gemv_w4_amd", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


# --------------------------------------------------------------------------
# The oracle's own pins
# --------------------------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128])
def test_oracle_whole_block_is_one_row(d):
    x = np.random.default_rng(d).standard_normal((16, d)).astype(np.float32)
    codes, scale, st = oracle.write_block_ref(np.full((16, d), 77, np.int8), np.float32(9.0), {r: x[r] for r in range(16)})
    rc, rs = oracle.quantize_rows_int8_ref(x.reshape(1, -1))
    assert np.array_equal(codes.reshape(1, -1), rc) and scale == rs[0] and st == 0


def test_oracle_block_grows_and_begins_anew():
    d = 64
    x = np.zeros((16, d), np.float32)
    x[:, 0] = [1, 2, 2, 3, 1, 12.7] + [1] * 10
    codes, scale = np.full((16, d), 5, np.int8), np.float32(np.nan)
    steps = []
    for r in range(16):
        codes, scale, _ = oracle.write_block_ref(codes, scale, {r: x[r]})
        steps.append(float(scale))
    assert steps == [float(np.float32(v / 127)) for v in [1, 2, 2, 3, 3] + [12.7] * 11]
    assert codes[:, 0].tolist() == [10, 20, 20, 30, 10, 127] + [10] * 10
    assert np.all(codes[:, 1:] == 0)
    again, scale, _ = oracle.write_block_ref(codes, scale, {0: x[0]})   # the first row: anew, the others as they were
    assert float(scale) == float(np.float32(1 / 127)) and again[0, 0] == 127 and np.array_equal(again[1:], codes[1:])
    # zeros, values that are not finite, scales that are none
    codes, scale, st = oracle.write_block_ref(codes, np.float32(-2.0), {3: np.full(d, np.nan), 4: np.zeros(d)})
    assert scale == 0 and st == 1 and np.all(codes[3:5] == 0)


def test_oracle_scores_reduce_to_plain_attention():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 4, 64)), rng.standard_normal((2, 30, 64)), rng.standard_normal((2, 30, 64))
    for window in (0, 7):
        a = oracle.attention_ref(q, k, v, 30, 0.125, window)
        b = oracle.attention_scores_ref(q, k, v, 30, 0.125, window)
        assert np.allclose(a[0], b[0], rtol=0, atol=1e-14) and np.allclose(a[1], b[1], rtol=0, atol=1e-14)
    # a prefix past every key is attention without a mask; a document's rows are those of the document alone
    full = oracle.attention_scores_ref(q, k, v, 30, 0.125, prefix=99)[0]
    last = oracle.attention_scores_ref(q[4:], k, v, 30, 0.125)[0]
    assert np.allclose(full[4], last[0], rtol=0, atol=1e-14)
    own = oracle.attention_scores_ref(q, k, v, 30, 0.125, first=np.full(5, 20), slopes=[1.0, 0.5, 0.25, 0.0])[0]
    alone = oracle.attention_scores_ref(q, k[:, 20:], v[:, 20:], 10, 0.125, slopes=[1.0, 0.5, 0.25, 0.0])[0]
    assert np.allclose(own, alone, rtol=0, atol=1e-14)
    assert np.all(oracle.attention_scores_ref(q, k, v, 30, 0.125, first=np.full(5, 30))[0] == 0)
