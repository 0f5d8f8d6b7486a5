"""Binding of the operators between the products of a decoder layer: the root-mean-square norm, the
gate, rotary positions with the write into a paged cache, its rows read back, block tables, and paged
attention.

Argument marshalling only, like the rest of the package; tensors have to be contiguous and on one
GPU, and a call runs on that GPU's current stream.  A decode step makes hundreds of these calls,
each a few microseconds long on the device, so an argument is checked in one expression and told
apart only when it is wrong.
"""

from __future__ import annotations

import ctypes

import torch

from . import W4_BF16, W4_F32, W4Rope, _check, _KVCacheStruct, _require, _ScoresStruct, lib

_FLOATS = (torch.float32, torch.bfloat16)
_F32, _BF16, _I32, _I64 = (torch.float32,), (torch.bfloat16,), (torch.int32,), (torch.int64,)
_F64, _U8, _I8 = (torch.float64,), (torch.uint8,), (torch.int8,)


def _want(t, dtypes, shape, name, index):
    """A contiguous tensor of one of the types on GPU ``index``, of that shape unless it is None."""
    try:
        if t.dtype in dtypes and t.get_device() == index and t.is_contiguous() and (shape is None or t.shape == shape):
            return
    except AttributeError:
        pass
    _require(t, dtypes, shape, name)
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _code(t):
    return W4_F32 if t.dtype is torch.float32 else W4_BF16


def _opt(t):
    return None if t is None else t.data_ptr()


def _status_ptr(status, index):
    if status is None:
        return None
    _want(status, _I32, None, "status", index)
    if status.numel() < 1:
        raise ValueError("status must hold one element")
    return status.data_ptr()


_FUNCTIONS = {}
_current_device = getattr(torch._C, "_cuda_getDevice", None)             # neither in a build without GPUs
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(name, index, *args):
    """Run an entry point on GPU ``index`` and its current stream."""
    fn = _FUNCTIONS.get(name)
    if fn is None:
        fn = _FUNCTIONS[name] = getattr(lib(), name)
    if index == _current_device():
        status = fn(*args, _current_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _current_stream(index))
    if status:
        _check(status, name)


def _rows_of(x, name):
    """x as [rows, values] on a GPU."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype not in _FLOATS or not x.is_contiguous():
        _require(x, _FLOATS, None, name)
    dim = x.dim()
    if dim == 2:
        return x
    if dim != 1:
        raise ValueError(f"{name} must be [rows, values]")
    return x.unsqueeze(0)


def _value_rows(y, out_dtype, shape, x, index):
    if y is None:
        if (out_dtype or torch.bfloat16) not in _FLOATS:
            raise TypeError(f"out_dtype is {out_dtype}")
        return torch.empty(shape, dtype=out_dtype or torch.bfloat16, device=x.device)
    _want(y, _FLOATS, shape, "y", index)
    return y


def _code_rows(codes, scales, dtypes, shape, x, index):
    if codes is None:
        codes = torch.empty(shape, dtype=dtypes[0], device=x.device)
    else:
        _want(codes, dtypes, shape, "codes", index)
    if scales is None:
        scales = torch.empty(shape[0], dtype=torch.float32, device=x.device)
    else:
        _want(scales, _F32, (shape[0],), "scales", index)
    return codes, scales


def _norm_args(x, weight, eps, residual, residual_out):
    x = _rows_of(x, "x")
    shape, index = x.shape, x.get_device()
    rows, K = shape
    _want(weight, _FLOATS, (K,), "weight", index)
    r = r_out = None
    rt = W4_F32
    if residual is not None:
        if residual.dim() == 1:
            residual = residual.unsqueeze(0)
        _want(residual, _FLOATS, shape, "residual", index)
        r, rt = residual.data_ptr(), _code(residual)
        r_out = r
        if residual_out is not None:
            if residual_out.dim() == 1:
                residual_out = residual_out.unsqueeze(0)
            _want(residual_out, (residual.dtype,), shape, "residual_out", index)
            r_out = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out without residual")
    return x, shape, index, (x.data_ptr(), _code(x), r, r_out, rt, weight.data_ptr(), _code(weight), eps, rows, K)


def w4_rmsnorm(x, weight, eps, residual=None, residual_out=None, y=None, out_dtype=None):
    """Root-mean-square norm of x [rows, K] (after adding ``residual``, which is updated in place
    unless ``residual_out`` is given); y [rows, K] bfloat16 by default."""
    x, shape, index, args = _norm_args(x, weight, eps, residual, residual_out)
    y = _value_rows(y, out_dtype, shape, x, index)
    _call("w4_rmsnorm", index, *args, y.data_ptr(), _code(y))
    return y


def _rmsnorm_codes(name, dtypes, x, weight, eps, residual, residual_out, codes, scales, status):
    x, shape, index, args = _norm_args(x, weight, eps, residual, residual_out)
    codes, scales = _code_rows(codes, scales, dtypes, shape, x, index)
    _call(name, index, *args, codes.data_ptr(), scales.data_ptr(), _status_ptr(status, index))
    return codes, scales


def w4_rmsnorm_fp8(x, weight, eps, residual=None, residual_out=None, codes=None, scales=None, status=None):
    """w4_rmsnorm quantized per row: E4M3 codes [rows, K] uint8 and scales [rows]."""
    return _rmsnorm_codes("w4_rmsnorm_fp8", _U8, x, weight, eps, residual, residual_out, codes, scales, status)


def w4_rmsnorm_int8(x, weight, eps, residual=None, residual_out=None, codes=None, scales=None, status=None):
    """w4_rmsnorm quantized per row: symmetric INT8 codes [rows, K] and steps [rows]."""
    return _rmsnorm_codes("w4_rmsnorm_int8", _I8, x, weight, eps, residual, residual_out, codes, scales, status)


def _gate_args(gate_up):
    x = _rows_of(gate_up, "gate_up")
    rows, width = x.shape
    if width % 2:
        raise ValueError("gate_up must be [rows, 2F]")
    F = width // 2
    return x, (rows, F), x.get_device(), (x.data_ptr(), _code(x), rows, F)


def w4_silu_mul(gate_up, y=None, out_dtype=None):
    """silu(gate) * up of gate_up [rows, 2F] (gate first); y [rows, F] bfloat16 by default."""
    x, shape, index, args = _gate_args(gate_up)
    y = _value_rows(y, out_dtype, shape, x, index)
    _call("w4_silu_mul", index, *args, y.data_ptr(), _code(y))
    return y


def _silu_mul_codes(name, dtypes, gate_up, codes, scales, status):
    x, shape, index, args = _gate_args(gate_up)
    codes, scales = _code_rows(codes, scales, dtypes, shape, x, index)
    _call(name, index, *args, codes.data_ptr(), scales.data_ptr(), _status_ptr(status, index))
    return codes, scales


def w4_silu_mul_fp8(gate_up, codes=None, scales=None, status=None):
    """w4_silu_mul quantized per row: E4M3 codes [rows, F] uint8 and scales [rows]."""
    return _silu_mul_codes("w4_silu_mul_fp8", _U8, gate_up, codes, scales, status)


def w4_silu_mul_int8(gate_up, codes=None, scales=None, status=None):
    """w4_silu_mul quantized per row: symmetric INT8 codes [rows, F] and steps [rows]."""
    return _silu_mul_codes("w4_silu_mul_int8", _I8, gate_up, codes, scales, status)


class W4KVCache:
    """A paged cache: k and v [pages, kv_heads, page_size, head_dim], bfloat16; uint8 (E4M3 codes)
    with float32 scales [pages, kv_heads, page_size]; or int8 with float32 scales [pages, kv_heads,
    page_size / 16].  Keeps its tensors alive."""

    BLOCK = 16                                                # rows of an int8 cache that share a scale
    _TYPES = {torch.bfloat16: 0, torch.uint8: 1, torch.int8: 3}

    def __init__(self, k, v, k_scales=None, v_scales=None):
        _require(k, (torch.bfloat16, torch.uint8, torch.int8), None, "k")
        if k.dim() != 4:
            raise ValueError("k must be [pages, kv_heads, page_size, head_dim]")
        index = k.get_device()
        _want(v, (k.dtype,), k.shape, "v", index)
        if k.dtype != torch.bfloat16:
            if k.dtype == torch.int8 and k.shape[2] % self.BLOCK:
                raise ValueError("page_size must be a multiple of 16")
            shape = self._scales_shape(k.shape, k.dtype)
            _want(k_scales, _F32, shape, "k_scales", index)
            _want(v_scales, _F32, shape, "v_scales", index)
        elif k_scales is not None or v_scales is not None:
            raise ValueError("a bfloat16 cache has no scales")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self.device, self._index = k.device, index
        self._c = _KVCacheStruct(k.data_ptr(), v.data_ptr(), _opt(k_scales), _opt(v_scales), self.pages,
                                 self.page_size, self.kv_heads, self.head_dim, self._TYPES[k.dtype])
        self._ref = ctypes.byref(self._c)

    @classmethod
    def _scales_shape(cls, shape, dtype):
        return (*shape[:2], shape[2] // cls.BLOCK if dtype == torch.int8 else shape[2])

    @classmethod
    def empty(cls, pages, page_size, kv_heads, head_dim, fp8=False, device="cuda", int8=False):
        """A cache of that shape (zeros)."""
        if fp8 and int8:
            raise ValueError("a cache holds one type")
        shape = (pages, kv_heads, page_size, head_dim)
        dtype = torch.uint8 if fp8 else torch.int8 if int8 else torch.bfloat16
        kv = [torch.zeros(shape, dtype=dtype, device=device) for _ in range(2)]
        if dtype == torch.bfloat16:
            return cls(*kv)
        scale = torch.ones if fp8 else torch.zeros
        return cls(*kv, *[scale(cls._scales_shape(shape, dtype), dtype=torch.float32, device=device) for _ in range(2)])


def w4_rope_cache(qkv, cache: W4KVCache, positions, slots, rope: W4Rope, freqs, q=None, status=None):
    """Rotate the rows of the fused q|k|v product qkv [T, (heads + 2 kv_heads) * head_dim] and store
    K and V at ``slots``; returns q [T, heads, head_dim] bfloat16.  ``freqs``: float64 device tensor
    of w4_rope_frequencies.  Rows with a negative slot are left out (of q too)."""
    x = _rows_of(qkv, "qkv")
    index = cache._index
    T, width = x.shape
    d = cache.head_dim
    heads = width // d - 2 * cache.kv_heads
    if width % d or heads < 1:
        raise ValueError("qkv must be [T, (heads + 2 kv_heads) * head_dim]")
    if x.get_device() != index:
        raise ValueError(f"cache is on {cache.device}, expected {x.device}")
    _want(positions, _I32, (T,), "positions", index)
    _want(slots, _I64, (T,), "slots", index)
    _want(freqs, _F64, (rope.rotary_dim // 2,), "freqs", index)
    if q is None:
        q = torch.empty((T, heads, d), dtype=torch.bfloat16, device=x.device)
    else:
        _want(q, _BF16, (T, heads, d), "q", index)
    _call("w4_rope_cache", index, x.data_ptr(), _code(x), T, heads, cache._ref, positions.data_ptr(),
          slots.data_ptr(), ctypes.byref(rope), freqs.data_ptr(), q.data_ptr(), _status_ptr(status, index))
    return q


def w4_cache_write(qkv, cache: W4KVCache, slots, q=None, status=None):
    """w4_rope_cache without rotation: store K and V of qkv [T, (heads + 2 kv_heads) * head_dim] at
    ``slots``; returns q [T, heads, head_dim] bfloat16, or None where qkv holds no query heads."""
    x = _rows_of(qkv, "qkv")
    index = cache._index
    T, width = x.shape
    d = cache.head_dim
    heads = width // d - 2 * cache.kv_heads
    if width % d or heads < 0:
        raise ValueError("qkv must be [T, (heads + 2 kv_heads) * head_dim]")
    if x.get_device() != index:
        raise ValueError(f"cache is on {cache.device}, expected {x.device}")
    _want(slots, _I64, (T,), "slots", index)
    if heads == 0:
        if q is not None:
            raise ValueError("q without query heads in qkv")
    elif q is None:
        q = torch.empty((T, heads, d), dtype=torch.bfloat16, device=x.device)
    else:
        _want(q, _BF16, (T, heads, d), "q", index)
    _call("w4_cache_write", index, x.data_ptr(), _code(x), T, heads, cache._ref, slots.data_ptr(), _opt(q),
          _status_ptr(status, index))
    return q


def w4_cache_read(cache: W4KVCache, slots, out=None, out_dtype=None, status=None):
    """Rows of the cache at ``slots`` [n] as values [n, 2 kv_heads * head_dim] (key heads, value heads; what
    w4_cache_write takes), bfloat16 by default.  Rows of slots that are negative or past the cache are left."""
    index = cache._index
    _want(slots, _I64, None, "slots", index)
    if slots.dim() != 1:
        raise ValueError("slots must be [n]")
    shape = (slots.numel(), 2 * cache.kv_heads * cache.head_dim)
    if out is None:
        if (out_dtype or torch.bfloat16) not in _FLOATS:
            raise TypeError(f"out_dtype is {out_dtype}")
        out = torch.empty(shape, dtype=out_dtype or torch.bfloat16, device=cache.device)
    else:
        _want(out, _FLOATS, shape, "out", index)
    _call("w4_cache_read", index, cache._ref, slots.data_ptr(), shape[0], out.data_ptr(), _code(out),
          _status_ptr(status, index))
    return out


def w4_block_tables(new_lens, lens, free_pages, free_count, block_table, page_size, tokens=None, lens_out=None,
                    free_count_out=None, cu_q=None, positions=None, slots=None, status=None):
    """Place the new tokens of a batch in pages; returns (cu_q, positions, slots).

    ``lens`` and ``free_count`` are updated in place unless ``lens_out`` / ``free_count_out`` are
    given; ``block_table`` is.  ``tokens``: places of positions and slots where those are not given."""
    _require(new_lens, _I32, None, "new_lens")
    index = new_lens.get_device()
    if new_lens.dim() != 1:
        raise ValueError("new_lens must be [B]")
    B = new_lens.numel()
    each = (B,)
    if positions is None or slots is None:
        if positions is not None:
            tokens = positions.numel()
        elif slots is not None:
            tokens = slots.numel()
        elif tokens is None:
            raise ValueError("tokens is needed where positions and slots are not given")
        device = new_lens.device
        positions = torch.empty(tokens, dtype=torch.int32, device=device) if positions is None else positions
        slots = torch.empty(tokens, dtype=torch.int64, device=device) if slots is None else slots
    if cu_q is None:
        cu_q = torch.empty(B + 1, dtype=torch.int32, device=new_lens.device)
    else:
        _want(cu_q, _I32, (B + 1,), "cu_q", index)
    _want(lens, _I32, each, "lens", index)
    _want(free_pages, _I32, None, "free_pages", index)
    _want(free_count, _I32, (1,), "free_count", index)
    _want(block_table, _I32, None, "block_table", index)
    if lens_out is None:
        lens_out = lens
    else:
        _want(lens_out, _I32, each, "lens_out", index)
    if free_count_out is None:
        free_count_out = free_count
    else:
        _want(free_count_out, _I32, (1,), "free_count_out", index)
    table_shape = block_table.shape
    if len(table_shape) != 2 or table_shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")
    _want(positions, _I32, None, "positions", index)
    T = positions.numel()
    _want(slots, _I64, positions.shape, "slots", index)
    _call("w4_block_tables", index, new_lens.data_ptr(), lens.data_ptr(), B, free_pages.data_ptr(),
          free_pages.numel(), free_count.data_ptr(), lens_out.data_ptr(), free_count_out.data_ptr(),
          block_table.data_ptr(), table_shape[1], page_size, cu_q.data_ptr(), positions.data_ptr(),
          slots.data_ptr(), T, _status_ptr(status, index))
    return cu_q, positions, slots


def w4_paged_attention_workspace_bytes(T: int, heads: int, cache: W4KVCache, B: int, max_pages: int) -> int:
    return int(lib().w4_paged_attention_workspace_bytes(T, heads, cache._ref, B, max_pages))


def w4_paged_attention(q, cache: W4KVCache, block_table, cu_q, lens, scale, window=0, o=None, workspace=None,
                       status=None):
    """Attention of q [T, heads, head_dim] (bfloat16) over the paged cache; returns o like q.

    ``cu_q`` [B + 1] and ``lens`` [B] as w4_block_tables gives them (lens counts the new tokens);
    rows of q behind cu_q[B] are left out of o.  The workspace is allocated where it is not given."""
    return _attend("w4_paged_attention", (), q, cache, block_table, cu_q, lens, scale, window, o, workspace, status)


class W4Scores:
    """Scores and keys other than the plain causal ones: scores capped at ``cap``; ``slopes`` [heads] float32 of
    a bias by distance; ``first_keys`` [T] int32, the first key that each row of the batch sees (of its
    document); ``prefix_lens`` [B] int32, tokens at the start of each request that all its rows see.  Keeps its
    tensors alive."""

    def __init__(self, cap=0.0, slopes=None, first_keys=None, prefix_lens=None):
        for t, dtypes, name in ((slopes, _F32, "slopes"), (first_keys, _I32, "first_keys"), (prefix_lens, _I32, "prefix_lens")):
            if t is not None:
                _require(t, dtypes, None, name)
        self.cap, self.slopes, self.first_keys, self.prefix_lens = cap, slopes, first_keys, prefix_lens
        self._c = _ScoresStruct(cap, 0, _opt(slopes), _opt(first_keys), _opt(prefix_lens))
        self._ref = ctypes.byref(self._c)

    def __setattr__(self, name, value):
        if "_ref" in self.__dict__:                           # its record would still name the old ones
            raise AttributeError("a W4Scores keeps what it was made with: write into its tensors or make another")
        super().__setattr__(name, value)


def w4_paged_attention_scores(q, cache: W4KVCache, block_table, cu_q, lens, scale, scores: W4Scores, window=0, o=None,
                              workspace=None, status=None):
    """w4_paged_attention with the scores and keys that ``scores`` asks for; the workspace is of the same size."""
    index = cache._index
    _want(q, _BF16, None, "q", index)
    if scores.slopes is not None:
        _want(scores.slopes, _F32, tuple(q.shape[1:2]), "slopes", index)
    if scores.first_keys is not None:
        _want(scores.first_keys, _I32, tuple(q.shape[:1]), "first_keys", index)
    if scores.prefix_lens is not None:
        _want(scores.prefix_lens, _I32, tuple(lens.shape), "prefix_lens", index)
    return _attend("w4_paged_attention_scores", (scores._ref,), q, cache, block_table, cu_q, lens, scale, window, o, workspace,
                   status)


def _attend(name, scores, q, cache, block_table, cu_q, lens, scale, window, o, workspace, status):
    index = cache._index
    _want(q, _BF16, None, "q", index)
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.head_dim:
        raise ValueError("q must be [T, heads, head_dim]")
    T, heads, _ = shape
    _want(block_table, _I32, None, "block_table", index)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = block_table.shape
    _want(cu_q, _I32, (B + 1,), "cu_q", index)
    _want(lens, _I32, (B,), "lens", index)
    if o is None:
        o = torch.empty_like(q)
    else:
        _want(o, _BF16, shape, "o", index)
    if workspace is None:
        need = w4_paged_attention_workspace_bytes(T, heads, cache, B, max_pages)
        workspace = torch.empty(need, dtype=torch.uint8, device=cache.device) if need else None
    else:
        _want(workspace, _U8, None, "workspace", index)
    _call(name, index, q.data_ptr(), T, heads, cache._ref, block_table.data_ptr(),
          max_pages, cu_q.data_ptr(), lens.data_ptr(), B, scale, window, *scores, o.data_ptr(), _opt(workspace),
          0 if workspace is None else workspace.numel(), _status_ptr(status, index))
    return o
