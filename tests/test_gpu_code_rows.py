"""8-bit rows with values that are not finite: the norm, the gate and the cache write give the bytes
that the row quantizers give for the binary32 rows (0x7F, E4M3's NaN, is never written)."""

import numpy as np
import pytest
import torch

import dequant_gemv_w4_amd as w4
from test_gpu_operators import BF, DEV, F32, _dev, _say

pytestmark = pytest.mark.gpu
QUANTIZE = {"fp8": w4.w4_fp8_quantize_rows, "int8": w4.w4_int8_quantize_rows}


def _spoiled(rows, k, seed):
    """Rows with a NaN, an infinity of either sign, several of them, nothing else, and none."""
    x = np.random.default_rng(seed).standard_normal((rows, k)).astype(np.float32)
    x[1, 3] = np.nan
    x[2, k - 1] = np.inf
    x[3, 0], x[3, 9], x[3, k // 2] = np.nan, -np.inf, np.nan
    x[4] = np.nan
    x[5, 64:72] = np.nan
    x[6] = 0.0
    x[6, 17] = -np.nan
    return x


def _same(got, y, kind, what):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    codes, scales = QUANTIZE[kind](y, status=st)
    assert torch.equal(got[0], codes), f"{what}: {int((got[0] != codes).sum())} codes differ"
    assert torch.equal(got[1].view(torch.int32), scales.view(torch.int32)), what
    assert int(st) == 1
    if kind == "fp8":
        assert not bool(((got[0] & 0x7F) == 0x7F).any())


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("rows,k", [(8, 256), (8, 2176), (600, 1024)])
def test_gate_rows(kind, rows, k):
    _say(f"gate rows {kind} {rows}x{k}")
    u = _spoiled(rows, k, 3)
    x = _dev(np.concatenate([np.full((rows, k), 64.0, np.float32), u], 1))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = (w4.w4_silu_mul_fp8 if kind == "fp8" else w4.w4_silu_mul_int8)(x, status=st)
    assert int(st) == 1
    _same(got, w4.w4_silu_mul(x, out_dtype=F32), kind, "gate")


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("rows,k", [(8, 256), (8, 2176), (600, 1024)])
def test_norm_rows(kind, rows, k):
    _say(f"norm rows {kind} {rows}x{k}")
    x = _dev(_spoiled(rows, k, 4))
    w = torch.ones(k, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = (w4.w4_rmsnorm_fp8 if kind == "fp8" else w4.w4_rmsnorm_int8)(x, w, 1e-5, status=st)
    assert int(st) == 1
    _same(got, w4.w4_rmsnorm(x, w, 1e-5, out_dtype=F32), kind, "norm")
    # a weight that is not finite leaves finite values beside it in every row
    x = torch.randn(rows, k, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(BF)
    for at, value in ((5, "nan"), (k - 3, "inf")):
        w[at] = float(value)
        got = (w4.w4_rmsnorm_fp8 if kind == "fp8" else w4.w4_rmsnorm_int8)(x, w, 1e-5)
        _same(got, w4.w4_rmsnorm(x, w, 1e-5, out_dtype=F32), kind, "weight")


def test_cache_rows():
    heads, kv, d, T, page = 3, 3, 128, 8, 16
    x = _spoiled(T, (heads + 2 * kv) * d, 6)
    x[:, (heads + kv) * d:] = _spoiled(T * kv, d, 7).reshape(T, kv * d)
    cache = w4.W4KVCache.empty(1, page, kv, d, fp8=True, device=DEV)
    spec = w4.W4Rope.make(64)
    freqs, _ = w4.w4_rope_frequencies(spec, DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    w4.w4_rope_cache(_dev(x), cache, torch.zeros(T, dtype=torch.int32, device=DEV), torch.arange(T, device=DEV), spec, freqs, status=st)
    assert int(st) == 1
    for part, codes, scales in ((x[:, heads * d: (heads + kv) * d], cache.k, cache.k_scales), (x[:, (heads + kv) * d:], cache.v, cache.v_scales)):
        y = _dev(np.ascontiguousarray(part).reshape(T * kv, d))   # position 0: the rows as they are
        rc, rs = w4.w4_fp8_quantize_rows(y)
        got = codes[0, :, :T].transpose(0, 1).reshape(T * kv, d)
        gs = scales[0, :, :T].t().reshape(-1)
        # keys: a pair of which one is not finite turns to two that are not (x * cos 0 - NaN * sin 0), values not
        clean = torch.isfinite(y).all(1) if codes is cache.k else torch.ones(T * kv, dtype=torch.bool, device=DEV)
        assert torch.equal(got[clean], rc[clean]) and torch.equal(gs[clean].view(torch.int32), rs[clean].view(torch.int32))
        assert not bool(((got & 0x7F) == 0x7F).any())
