"""Host-side checks of the operators between a layer's products (no GPU needed): refusals before
any device work, sizes in closed form, rotary frequencies, and the oracle of the block tables.
No call here passes validation, so no kernel is launched.
"""

import ctypes
import math

import numpy as np
import pytest

import dequant_gemv_w4_amd as w4
import oracle

NULL = ctypes.c_void_p(None)
OK_ADDR = 0x100000


def f(addr=OK_ADDR):
    return ctypes.c_void_p(addr)


def cache(**kw):
    d = dict(k=OK_ADDR, v=OK_ADDR, k_scales=None, v_scales=None, pages=10, page_size=16, kv_heads=2, head_dim=128, type=0)
    d.update(kw)
    return ctypes.byref(w4._KVCacheStruct(**d))


def rope(*a, **kw):
    return ctypes.byref(w4.W4Rope.make(*a, **kw))


@pytest.mark.parametrize("kind", ["plain", "fp8", "int8"])
def test_norm_refusals(kind):
    L = w4.lib()
    fn = {"plain": L.w4_rmsnorm, "fp8": L.w4_rmsnorm_fp8, "int8": L.w4_rmsnorm_int8}[kind]

    def call(x=f(), xt=1, r=NULL, ro=NULL, rt=0, w=f(), wt=1, eps=1e-5, rows=4, k=256, y=f(), last=None):
        tail = (y, 1, NULL) if kind == "plain" else (y, f() if last is None else last, NULL, NULL)
        return fn(x, xt, r, ro, rt, w, wt, eps, rows, k, *tail)

    assert call(x=NULL) == 1 and call(w=NULL) == 1 and call(y=NULL) == 1
    assert call(r=f()) == 1 and call(ro=f()) == 1             # residual and residual_out go together
    assert call(xt=2) == 4 and call(wt=-1) == 4 and call(r=f(), ro=f(), rt=3) == 4
    assert call(rows=0) == 2 and call(rows=1 << 31) == 2
    assert call(k=64) == 2 and call(k=200) == 2 and call(k=65536 + 128) == 2
    for eps in (0.0, -1e-5, math.inf, math.nan):
        assert call(eps=eps) == 10
    off = f(OK_ADDR + 8)
    assert call(x=off) == 3 and call(w=off) == 3 and call(y=off) == 3 and call(r=off, ro=f()) == 3 and call(r=f(), ro=off) == 3
    if kind == "plain":
        assert L.w4_rmsnorm(f(), 1, NULL, NULL, 0, f(), 1, 1e-5, 4, 256, f(), 7, NULL) == 4
    else:
        assert call(last=NULL) == 1 and call(last=f(OK_ADDR + 2)) == 3


@pytest.mark.parametrize("kind", ["plain", "fp8", "int8"])
def test_gate_refusals(kind):
    L = w4.lib()
    fn = {"plain": L.w4_silu_mul, "fp8": L.w4_silu_mul_fp8, "int8": L.w4_silu_mul_int8}[kind]

    def call(x=f(), xt=1, rows=4, k=256, y=f(), last=None):
        tail = (y, 1, NULL) if kind == "plain" else (y, f() if last is None else last, NULL, NULL)
        return fn(x, xt, rows, k, *tail)

    assert call(x=NULL) == 1 and call(y=NULL) == 1 and call(xt=9) == 4
    assert call(rows=0) == 2 and call(k=0) == 2 and call(k=129) == 2 and call(k=1 << 17) == 2
    assert call(x=f(OK_ADDR + 4)) == 3 and call(y=f(OK_ADDR + 4)) == 3
    if kind != "plain":
        assert call(last=NULL) == 1


BAD_CACHES = [(dict(type=2), 5), (dict(head_dim=96), 5), (dict(head_dim=0), 5), (dict(page_size=8), 5), (dict(page_size=48), 5),
              (dict(page_size=8192), 5), (dict(page_size=-16), 5), (dict(kv_heads=0), 2), (dict(kv_heads=1025), 2), (dict(pages=0), 2),
              (dict(pages=(1 << 31) - 1, page_size=4096, kv_heads=1024), 2),
              (dict(k=None), 1), (dict(v=None), 1), (dict(k=OK_ADDR + 8), 3), (dict(type=1, v_scales=OK_ADDR), 1),
              (dict(type=1, k_scales=OK_ADDR, v_scales=OK_ADDR + 2), 3)]


def test_rope_cache_refusals():
    L = w4.lib()

    def call(x=f(), xt=1, T=3, heads=4, c=None, pos=f(), slots=f(), r=None, fr=f(), q=f()):
        return L.w4_rope_cache(x, xt, T, heads, c or cache(), pos, slots, r or rope(64), fr, q, NULL, NULL)

    for name in ("x", "pos", "slots", "fr", "q"):
        assert call(**{name: NULL}) == 1, name
    assert L.w4_rope_cache(f(), 1, 3, 4, None, f(), f(), rope(64), f(), f(), NULL, NULL) == 1
    assert L.w4_rope_cache(f(), 1, 3, 4, cache(), f(), f(), None, f(), f(), NULL, NULL) == 1
    assert call(xt=2) == 4
    assert call(T=0) == 2 and call(T=(1 << 22) + 1) == 2 and call(heads=3) == 2 and call(heads=0) == 2
    assert call(T=1 << 22, heads=16) == 2                     # T * heads past its limit
    assert call(T=1, heads=65538) == 2
    for kw, status in BAD_CACHES:
        assert call(c=cache(**kw)) == status, kw
    assert call(r=rope(24)) == 5 and call(r=rope(0)) == 5 and call(r=rope(144)) == 5
    assert call(c=cache(head_dim=64), r=rope(80)) == 2
    assert call(r=rope(64, base=1.0)) == 10 and call(r=rope(64, scaling="linear", factor=0.5)) == 10
    assert call(x=f(OK_ADDR + 8)) == 3 and call(q=f(OK_ADDR + 8)) == 3 and call(slots=f(OK_ADDR + 4)) == 3
    assert call(fr=f(OK_ADDR + 4)) == 3 and call(pos=f(OK_ADDR + 2)) == 3


def test_rope_records():
    L = w4.lib()
    out = (ctypes.c_double * 64)()

    def call(r):
        return L.w4_rope_frequencies(ctypes.byref(r), out, None)

    R = w4.W4Rope.make
    assert call(R(64)) == 0
    assert L.w4_rope_frequencies(None, out, None) == 1 and L.w4_rope_frequencies(ctypes.byref(R(64)), None, None) == 1
    bad = R(64)
    bad.scaling = 4
    assert call(bad) == 5
    bad = R(64)
    bad.reserved = 1
    assert call(bad) == 5
    bad = R(64)
    bad.interleaved = 2
    assert call(bad) == 5
    for kw in (dict(base=math.nan), dict(base=math.inf), dict(base=0.5), dict(scaling="linear", factor=math.inf),
               dict(scaling="bands", factor=8, low=0.0, high=4.0), dict(scaling="bands", factor=8, low=4.0, high=4.0),
               dict(scaling="ramp", factor=8, original_positions=0), dict(scaling="ramp", factor=8, low=1, high=math.inf)):
        assert call(R(64, **kw)) == 10, kw
    with pytest.raises(ValueError):
        R(64, scaling="other")
    with pytest.raises(w4.W4Error):
        w4.w4_rope_frequencies(R(20))


@pytest.mark.parametrize("dim", [16, 64, 96, 128])
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="bands", factor=8.0, low=1.0, high=4.0, original=8192),
                                dict(scaling="ramp", factor=16.0, low=1.0, high=32.0, original=4096),
                                dict(scaling="ramp", factor=1.0, low=1.0, high=32.0, original=1),
                                dict(scaling="bands", factor=1.0, low=0.5, high=0.75, original=100)])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_rope_frequencies(dim, kw, base):
    ref, amp = oracle.rope_frequencies_ref(dim, base, **kw)
    args = dict(kw)
    if "original" in args:
        args["original_positions"] = args.pop("original")
    got, a = w4.w4_rope_frequencies(w4.W4Rope.make(dim, base, **args))
    assert len(got) == dim // 2
    # each side rounds a power, a quotient and a blend: a few units in the last place of binary64
    assert np.allclose(got, ref, rtol=1e-13, atol=0) and math.isclose(a, amp, rel_tol=1e-15)


def test_block_tables_refusals():
    L = w4.lib()
    names = ["new", "lens", "B", "free", "cap", "cin", "lout", "cout", "table", "max_pages", "page", "cu", "pos", "slots", "T"]

    def call(**kw):
        d = dict(new=f(), lens=f(), B=3, free=f(), cap=9, cin=f(), lout=f(), cout=f(), table=f(), max_pages=8, page=16, cu=f(), pos=f(),
                 slots=f(), T=5)
        d.update(kw)
        return L.w4_block_tables(*[d[n] for n in names], NULL, NULL)

    for n in ("new", "lens", "free", "cin", "lout", "cout", "table", "cu", "pos", "slots"):
        assert call(**{n: NULL}) == 1, n
        assert call(**{n: f(OK_ADDR + 2)}) == 3, n
    assert call(slots=f(OK_ADDR + 4)) == 3
    for page in (0, 8, 24, 8192, -16):
        assert call(page=page) == 5
    assert call(B=0) == 2 and call(B=4097) == 2 and call(T=0) == 2 and call(T=(1 << 22) + 1) == 2
    assert call(max_pages=0) == 2 and call(max_pages=(1 << 26) + 1) == 2 and call(cap=-1) == 2 and call(cap=1 << 31) == 2


def test_attention_refusals_and_workspace():
    L = w4.lib()

    def call(q=f(), T=3, heads=4, c=None, table=f(), max_pages=8, cu=f(), lens=f(), B=2, scale=0.1, window=0, o=f(), ws=f(), wb=1 << 40):
        return L.w4_paged_attention(q, T, heads, c or cache(), table, max_pages, cu, lens, B, scale, window, o, ws, wb, NULL, NULL)

    for n in ("q", "table", "cu", "lens", "o"):
        assert call(**{n: NULL}) == 1, n
    for kw, status in BAD_CACHES:
        assert call(c=cache(**kw)) == status, kw
    assert call(T=0) == 2 and call(heads=5) == 2 and call(heads=1) == 2 and call(T=1 << 22, heads=16) == 2
    assert call(B=0) == 2 and call(B=4097) == 2 and call(max_pages=0) == 2 and call(max_pages=(1 << 26) + 1) == 2
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=scale) == 10
    assert call(window=-1) == 10
    for n in ("q", "o", "ws"):
        assert call(**{n: f(OK_ADDR + 8)}) == 3, n
    for n in ("table", "cu", "lens"):
        assert call(**{n: f(OK_ADDR + 2)}) == 3, n

    def ws(T=1, heads=64, B=1, max_pages=1024, **kw):
        return L.w4_paged_attention_workspace_bytes(T, heads, cache(kv_heads=8, **kw), B, max_pages)

    # a long context and few rows: keys are split, and the parts of every tile of 32 rows kept
    assert ws() > 0 and ws() % (32 * (128 + 2) * 4) == 0
    assert ws(head_dim=64) * 130 == ws() * 66
    assert ws(max_pages=16) == 0                              # 256 keys are not worth splitting
    assert ws(T=4096, B=4096) == 0                            # workgroups enough
    assert ws(T=0) == 0 and ws(heads=7) == 0 and ws(page_size=20) == 0
    need = ws()
    args = dict(T=1, heads=64, c=cache(kv_heads=8), B=1, max_pages=1024)
    assert call(**args, wb=need - 1) == 7 and call(**args, ws=NULL) == 7


def test_status_text():
    assert w4.w4_status_string(10) == "argument value out of range"


def test_python_layer_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 256)
    with pytest.raises(ValueError):
        w4.w4_rmsnorm(x, x[0], 1e-5)
    with pytest.raises(ValueError):
        w4.w4_silu_mul_fp8(x)
    with pytest.raises(ValueError):
        w4.W4KVCache(torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16))
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        w4.w4_block_tables(i, i, i, i, i[None], 16, tokens=1)


def test_block_tables_oracle_by_hand():
    # pages of 16: request 0 has 20 tokens in 2 pages and gets 13 more (33: a third page), request 1
    # starts, request 2 cannot be served (one page left, it needs two), request 3 needs none
    table = [[7, 8, -1], [-1] * 3, [-1] * 3, [5, -1, -1]]
    cu, pos, slots, lens, left, out, status = oracle.block_tables_ref(
        [13, 1, 17, 2], [20, 0, 0, 4], [1, 2, 3, 4], 3, table, 16, 40)
    assert cu == [0, 13, 14, 31, 33] and lens == [33, 1, 0, 6] and left == 1 and status == 32
    assert out == [[7, 8, 3], [2, -1, -1], [-1] * 3, [5, -1, -1]]
    assert slots[:14] == [8 * 16 + i for i in range(4, 16)] + [3 * 16, 2 * 16]
    assert slots[14:31] == [-1] * 17 and slots[31:33] == [5 * 16 + 4, 5 * 16 + 5] and slots[33:] == [-1] * 7
    assert pos[12] == 32 and pos[13] == 0 and pos[31:33] == [4, 5]


def test_oracle_attention_and_rotation_by_hand():
    # equal scores: the mean of the visible values; a window of two keys; rows before the start see none
    v = np.arange(8.0).reshape(1, 4, 2)
    k = np.zeros((1, 4, 2))
    q = np.ones((2, 1, 2))
    o, _ = oracle.attention_ref(q, k, v, 4, 1.0)
    assert np.allclose(o[:, 0], [v[0, :3].mean(0), v[0].mean(0)])
    o, _ = oracle.attention_ref(q, k, v, 4, 1.0, window=2)
    assert np.allclose(o[:, 0], [v[0, 1:3].mean(0), v[0, 2:4].mean(0)])
    o, _ = oracle.attention_ref(q, k[:, :1], v[:, :1], 1, 1.0)
    assert np.allclose(o[0], 0) and np.allclose(o[1, 0], v[0, 0])
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    half = oracle.rope_ref(x, [1], np.array([math.pi / 2, math.pi]), 2.0, False)
    assert np.allclose(half, [[[-6.0, -4.0, 2.0, -8.0]]])
    inter = oracle.rope_ref(x, [1], np.array([math.pi / 2, math.pi]), 1.0, True)
    assert np.allclose(inter, [[[-2.0, 1.0, -3.0, -4.0]]])
