"""Requests over a shuffled paged cache of any type, for the GPU tests of the attention: what no request uses
holds NaN (codes of 127 and NaN scales in an INT8 cache)."""

from __future__ import annotations

import numpy as np
import torch

import dequant_gemv_w4_amd as w4
import oracle
from _util import to_np32

DEV = "cuda:0"
U32, UB = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


class Batch:
    def __init__(self, new, cached, heads, kv, d, page, kind, seed=0, pad=0, wide=0, qscale=1.0):
        rng = np.random.default_rng(seed)
        self.new, self.ctx = list(new), [n + c for n, c in zip(new, cached)]
        self.heads, self.kv, self.d, self.page, self.kind = heads, kv, d, page, kind
        need = [-(-c // page) for c in self.ctx]
        pages = sum(need) + 2
        order = rng.permutation(pages)
        self.table = np.full((len(need), max(max(need), 1) + wide), -1, np.int32)
        used = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[used: used + n]
            used += n
        self.keys, self.values = [], []
        shape = (pages, kv, page, d)
        raw, sc = {}, {n: None for n in "kv"}
        for n in "kv":
            if kind == "bf16":
                raw[n] = np.full(shape, np.nan, np.float32)
            elif kind == "fp8":
                raw[n], sc[n] = np.full(shape, 0x7F, np.uint8), np.full(shape[:3], np.nan, np.float32)
            else:
                raw[n], sc[n] = np.full(shape, 127, np.int8), np.full((pages, kv, page // 16), np.nan, np.float32)
        for b, c in enumerate(self.ctx):
            j = np.arange(c)
            pg, at = self.table[b, j // page], j % page
            for n, store in (("k", self.keys), ("v", self.values)):
                x = oracle.bf16_round((rng.standard_normal((c, kv, d)) * rng.uniform(0.3, 1, (1, kv, 1))).astype(np.float32))
                if kind == "bf16":
                    raw[n][pg, :, at] = x
                elif kind == "fp8":
                    codes, s = oracle.quantize_rows_fp8_ref(x.reshape(-1, d)) if c else (np.zeros((0, d), np.uint8), np.zeros(0, np.float32))
                    raw[n][pg, :, at] = codes.reshape(c, kv, d)
                    sc[n][pg, :, at] = s.reshape(c, kv)
                    x = oracle.E4M3_VALUES[codes].reshape(c, kv, d) * s.reshape(c, kv, 1).astype(np.float64)
                else:
                    blocks = -(-c // 16)
                    full = np.zeros((16 * blocks, kv, d), np.float32)
                    full[:c] = x
                    rows = full.reshape(blocks, 16, kv, d).transpose(0, 2, 1, 3).reshape(-1, 16 * d)
                    codes, s = oracle.quantize_rows_int8_ref(rows) if c else (np.zeros((0, 16 * d), np.int8), np.zeros(0, np.float32))
                    codes = codes.reshape(blocks, kv, 16, d).transpose(0, 2, 1, 3).reshape(-1, kv, d)[:c]
                    s = s.reshape(blocks, kv)
                    raw[n][pg, :, at] = codes
                    sc[n][self.table[b, 16 * np.arange(blocks) // page], :, np.arange(blocks) % (page // 16)] = s
                    x = codes * np.repeat(s, 16, 0)[:c, :, None].astype(np.float64)
                store.append(x.transpose(1, 0, 2))
        if kind == "bf16":
            self.cache = w4.W4KVCache(dev(raw["k"], BF), dev(raw["v"], BF))
        else:
            self.cache = w4.W4KVCache(dev(raw["k"]), dev(raw["v"]), dev(sc["k"]), dev(sc["v"]))
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.q = oracle.bf16_round((qscale * rng.standard_normal((int(self.cu[-1]) + pad, heads, d))).astype(np.float32))
        self.d_q, self.d_table, self.d_cu = dev(self.q, BF), dev(self.table), dev(self.cu)
        self.d_lens = dev(np.array(self.ctx, np.int32))
        self.scale = d ** -0.5
        self.status = 0

    def workspace(self, fill=0xFF):
        need = w4.w4_paged_attention_workspace_bytes(self.q.shape[0], self.heads, self.cache, len(self.new), self.table.shape[1])
        return torch.full((max(need, 1),), fill, dtype=torch.uint8, device=DEV)   # NaN in every part

    def run(self, window=0, scores=None, **kw):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        args = dict(o=torch.full(self.q.shape, 7.0, dtype=BF, device=DEV), workspace=self.workspace(), status=st, window=window)
        args.update(kw)
        given = (self.d_q, self.cache, self.d_table, self.d_cu, self.d_lens, self.scale)
        got = w4.w4_paged_attention(*given, **args) if scores is None else w4.w4_paged_attention_scores(*given, scores, **args)
        self.status = int(st)
        return got

    def check(self, got, window=0, what="", status=0, cap=0.0, slopes=None, first=None, prefix=None):
        """Against the oracle.  A weight p is off by 2^-8 (bfloat16) and its score's error: the product of d terms
        and its scalings, (d + 4) u of size = scale max sum |q| max |k|; with a cap 2^-19 of size; the bias and
        the exponent's argument 4 u of size + bias; exp2's result and the n / 8 partial sums as in the plain form."""
        assert self.status == status, f"{what}: status {self.status}"
        got = to_np32(got).astype(np.float64)
        for b, n in enumerate(self.new):
            if n == 0:
                continue
            s = slice(int(self.cu[b]), int(self.cu[b]) + n)
            q, ctx = self.q[s], self.ctx[b]
            ref, weight = oracle.attention_scores_ref(q, self.keys[b], self.values[b], ctx, self.scale, window, cap, slopes,
                                                      None if first is None else first[s], None if prefix is None else int(prefix[b]))
            size = self.scale * np.abs(q).sum(-1).max() * (np.abs(self.keys[b]).max() if ctx else 0)
            bias = 0.0 if slopes is None else np.abs(slopes).max() * ctx
            score = (self.d + 4) * U32 * size + (2.0 ** -19 * size if cap else 0.0) + 4 * U32 * (size + bias)
            tol = (UB + 2 * (score + (4 + ctx / 8) * U32)) * weight + UB * np.abs(ref) + 2.0 ** -100
            assert np.all(np.isfinite(got[s])), f"{what} request {b}: not finite"
            bad = np.abs(got[s] - ref) > tol
            if bad.any():
                i = np.unravel_index(np.argmax(np.abs(got[s] - ref) - tol), ref.shape)
                raise AssertionError(f"{what} request {b}: {bad.sum()} of {bad.size} off; at {i}: {got[s][i]!r} for {ref[i]!r}, tolerance {tol[i]:.3e}")
        assert np.all(got[int(self.cu[-1]):] == 7.0), f"{what}: rows behind the last request"
