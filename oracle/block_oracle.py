"""INT8 cache with a scale for each block of 16 rows, and attention with capped, biased or masked scores, in
binary64 on the CPU (tests only), row by row from their definitions.
"""

from __future__ import annotations

import numpy as np

BLOCK = 16
LEAST_SCALE = float(np.float32(2.0 ** -93 / 127))   # of those that a write leaves


def write_block_ref(codes, scale, rows):
    """One block of one kv head: codes [16, d] int8, scale binary32, rows {row: values [d] (binary32 values)} written
    at once.  Returns (codes, scale, status)."""
    codes, status = codes.copy(), 0
    y = {}
    for r, v in rows.items():
        v = np.asarray(v, dtype=np.float64)
        if not np.all(np.isfinite(v)):
            status = 1
        y[r] = np.where(np.isfinite(v), v, 0.0)
    most = max(np.abs(v).max() for v in y.values())
    if most < 2.0 ** -93:
        most = 0.0
    old = float(np.float32(scale))
    if 0 in rows or not np.isfinite(old) or old < LEAST_SCALE:
        old = 0.0
    step = most / 127
    if float(np.float32(step)) > old:
        scale = np.float32(step)
        if 0 not in rows:
            for r in range(BLOCK):
                if r not in rows:
                    codes[r] = np.rint(codes[r].astype(np.float64) / (step / old)).astype(np.int8) if old else 0
    else:
        scale, step = np.float32(old), old
    for r, v in y.items():
        codes[r] = np.rint(v / step).astype(np.int8) if step else 0
    return codes, scale, status


def write_rows_ref(codes, scales, x, slots):
    """A call: codes [pages, kv, page, d], scales [pages, kv, page / 16] (changed in place), x [T, kv, d], slots [T].
    Returns the status bits."""
    pages, kv, page, _ = codes.shape
    status, t = 0, 0
    while t < len(slots):
        slot = int(slots[t])
        if slot < 0:
            t += 1
            continue
        block, n = slot // BLOCK, 1
        while t + n < len(slots) and int(slots[t + n]) // BLOCK == block and int(slots[t + n]) >= 0:
            n += 1
        if slot >= pages * page:
            status |= 8
        else:
            p, i = slot // page, slot % page // BLOCK
            at = slice(BLOCK * i, BLOCK * (i + 1))
            for h in range(kv):
                rows = {int(slots[t + j]) % BLOCK: x[t + j, h] for j in range(n)}
                codes[p, h, at], scales[p, h, i], st = write_block_ref(codes[p, h, at], scales[p, h, i], rows)
                status |= st
        t += n
    return status


def block_values(codes, scales):
    """Values of a cache [pages, kv, page, d], binary64."""
    return codes.astype(np.float64) * np.repeat(scales.astype(np.float64), BLOCK, axis=2)[..., None]


def key_range_ref(pos, ctx, window=0, first=None, prefix=None):
    """[lo, hi] of the row at position pos."""
    hi = pos if prefix is None else max(pos, min(prefix, ctx) - 1)
    lo = max(0, first if first is not None else 0, pos - window + 1 if window else 0)
    return lo, hi


def attention_scores_ref(q, keys, values, ctx, scale, window=0, cap=0.0, slopes=None, first=None, prefix=None):
    """One request: q [n, heads, d] at positions ctx - n .. ctx - 1, keys and values [kv_heads, ctx, d], first [n],
    prefix a number.  Returns (o, weight) as attention_ref."""
    n, heads, d = q.shape
    group = heads // keys.shape[0]
    o, w = np.zeros((n, heads, d)), np.zeros((n, heads, d))
    for t in range(n):
        pos = ctx - n + t
        lo, hi = key_range_ref(pos, ctx, window, None if first is None else int(first[t]), prefix)
        if hi < lo or ctx == 0:
            continue
        j = np.arange(lo, hi + 1)
        for h in range(heads):
            z = keys[h // group, lo: hi + 1].astype(np.float64) @ q[t, h].astype(np.float64) * scale
            if cap:
                z = cap * np.tanh(z / cap)
            if slopes is not None:
                z = z - float(slopes[h]) * np.abs(pos - j)
            p = np.exp(z - z.max())
            v = values[h // group, lo: hi + 1].astype(np.float64)
            o[t, h] = p @ v / p.sum()
            w[t, h] = p @ np.abs(v) / p.sum()
    return o, w
