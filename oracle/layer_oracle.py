"""Operators between a decoder layer's products, in binary64 on the CPU (tests only).

Root-mean-square norm, the gate, rotary positions, block tables and attention, each from its
definition; block tables request by request in plain Python.
"""

from __future__ import annotations

import math

import numpy as np


def bf16_round(x: np.ndarray) -> np.ndarray:
    """binary32 values rounded to bfloat16 (nearest, halves to even), as binary32."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = (u + 0x7FFF + ((u >> np.uint64(16)) & np.uint64(1))) & np.uint64(0xFFFF0000)
    out = r.astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), out)


def residual_sum_ref(x: np.ndarray, r: np.ndarray, bf16: bool) -> np.ndarray:
    """x + r in one binary32 addition, rounded to the residual's type."""
    h = x.astype(np.float32) + r.astype(np.float32)
    return bf16_round(h) if bf16 else h


def rmsnorm_ref(h: np.ndarray, weight: np.ndarray, eps: float) -> np.ndarray:
    h = h.astype(np.float64)
    s = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + float(np.float32(eps)))
    return h * s * weight.astype(np.float64)


def silu_mul_ref(gate_up: np.ndarray) -> np.ndarray:
    f = gate_up.shape[1] // 2
    g, u = gate_up[:, :f].astype(np.float64), gate_up[:, f:].astype(np.float64)
    t = np.exp(-np.abs(g))
    with np.errstate(invalid="ignore"):                      # -inf * 0
        return np.where(g < 0, g * t, g) / (1.0 + t) * u


def rope_frequencies_ref(rotary_dim, base, scaling="none", factor=1.0, low=1.0, high=4.0, original=1):
    """(angles per position, amplitude)."""
    out = []
    for i in range(rotary_dim // 2):
        f = math.exp(-2.0 * i / rotary_dim * math.log(base))
        if scaling == "linear":
            f = f / factor
        elif scaling == "bands":
            wave = 2 * math.pi / f
            if wave >= original / low:
                f = f / factor
            elif wave > original / high:
                k = (original / wave - low) / (high - low)
                f = (1 - k) * f / factor + k * f
        elif scaling == "ramp":
            def dim(turns):
                return rotary_dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
            a, b = math.floor(dim(high)), math.ceil(dim(low))
            if b < 0:
                r = 1.0                                      # the ramp ends ahead of every pair
            elif a > rotary_dim - 1:
                r = 0.0                                      # begins behind every pair
            else:
                a, b = max(a, 0), min(b, rotary_dim - 1)
                r = min(max((i - a) / (b - a if b > a else 0.001), 0.0), 1.0)
            f = f / factor * r + f * (1 - r)
        out.append(f)
    return np.array(out), 1.0 + 0.1 * math.log(factor) if scaling == "ramp" else 1.0


def rope_ref(x: np.ndarray, positions, freqs, amplitude, interleaved) -> np.ndarray:
    """x [T, heads, d]: the first 2 * len(freqs) elements of each head turned."""
    x = x.astype(np.float64).copy()
    half = len(freqs)
    z = amplitude * np.exp(1j * np.outer(np.asarray(positions, dtype=np.float64), freqs))[:, None, :]
    i0 = 2 * np.arange(half) if interleaved else np.arange(half)
    i1 = i0 + 1 if interleaved else i0 + half
    w = (x[..., i0] + 1j * x[..., i1]) * z
    x[..., i0], x[..., i1] = w.real, w.imag
    return x


def block_tables_ref(new_lens, lens, free_pages, free_count, table, page, tokens):
    """(cu_q, positions, slots, lens_out, free_count_out, table_out, status)."""
    table = [list(map(int, row)) for row in table]
    count = min(max(int(free_count), 0), len(free_pages))
    positions, slots = [0] * tokens, [-1] * tokens
    cu, out, status, taken = [0], [], 0, 0
    for b, (n, have) in enumerate(zip(map(int, new_lens), map(int, lens))):
        start = cu[-1]
        cu.append(start + max(n, 0))
        out.append(have)
        if n < 0 or have < 0:
            status |= 16
            continue
        own = -(-have // page)
        need = -(-(have + n) // page) - own
        if own + need > len(table[b]):
            status |= 16 if start + n > tokens else 32
            continue
        if start + n > tokens:
            status |= 16
            continue
        if need and taken + need > count:
            status |= 32
            continue
        for i in range(need):
            table[b][own + i] = int(free_pages[count - 1 - taken - i])
        taken += need
        for i in range(n):
            p = have + i
            positions[start + i] = p
            at = table[b][p // page]
            slots[start + i] = at * page + p % page if at >= 0 else -1
        out[b] = have + n
    return [min(c, tokens) for c in cu], positions, slots, out, count - taken, table, status


def attention_ref(q, keys, values, ctx, scale, window=0):
    """One request: q [n, heads, d] at positions ctx - n .. ctx - 1, keys and values
    [kv_heads, ctx, d].  Returns (o, weight): o [n, heads, d] and sum_j p_j |v_j| / sum_j p_j."""
    n, heads, d = q.shape
    kv = keys.shape[0]
    o = np.zeros((n, heads, d))
    w = np.zeros((n, heads, d))
    if ctx == 0:
        return o, w
    pos = ctx - n + np.arange(n)[:, None]
    j = np.arange(ctx)[None, :]
    seen = j <= pos
    if window:
        seen &= j > pos - window
    some = seen.any(1)
    for h in range(heads):
        k, v = keys[h // (heads // kv)].astype(np.float64), values[h // (heads // kv)].astype(np.float64)
        z = np.where(seen, (q[:, h].astype(np.float64) @ k.T) * scale, -np.inf)
        m = np.where(some, z.max(1), 0.0)[:, None]
        p = np.where(seen, np.exp(z - m), 0.0)
        total = np.where(some, p.sum(1), 1.0)[:, None]
        o[:, h] = p @ v / total
        w[:, h] = p @ np.abs(v) / total
    return o, w
