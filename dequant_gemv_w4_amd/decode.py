"""A decode step: every quantized matrix of a model multiplied once by its activation rows.

Decode reads each weight once per generated token, so the step time is bounded
below by (weight bytes) / (HBM bandwidth) (page "Weight quantization", sections
"Complexity and constants" and "Efficiency"; page "Quantization" › "The idea in
one minute").  ``DecodeStep`` issues the w4_gemv calls of such a step back to
back on one stream and can capture them once into a graph, so replaying a step
costs a single launch from the host.

``DecoderStep`` runs whole decoder layers: the products with the norm, the rotary cache write, the
paged attention and the gate between them, for a batch that mixes prompts, chunks of prompts and
single tokens.  It keeps its buffers, so a step allocates nothing and can be captured too.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

from . import W4_BF16, W4_F32, W4Error, lib, w4_fp8_gemm, w4_fp8_quantize_rows, w4_gemm, w4_gemm_workspace_bytes
from . import w4_gemv, w4_int8_gemm, w4_int8_quantize_rows, w4_rope_frequencies


@dataclass
class GemvCall:
    prepared: object   # uint8 tensor from w4_prepare (or w4_prepare_fmt)
    n: int
    k: int
    x: object          # [M, K] bf16 or f32 tensor
    y: object          # [M, N] f32 or bf16 tensor
    fmt: object = None  # W4Format of the prepared layout; None: the canonical format

    def algorithmic_bytes(self) -> int:
        """Bytes the method must move: codes, scales and zeros as the format stores them
        (canonical: fp16 scales and byte zeros per 128 inputs), activations, outputs."""
        m = self.x.shape[0]
        group, zero_bits = (128, 8) if self.fmt is None else (self.fmt.group, self.fmt.zero_bits)
        groups = self.n * self.k // group
        return (self.n * self.k // 2 + groups * 2 + (groups * zero_bits + 7) // 8
                + m * self.k * self.x.element_size() + m * self.n * self.y.element_size())


class DecodeStep:
    def __init__(self, calls: list[GemvCall]):
        import torch
        self.calls = calls
        self._graph = None
        L = lib()
        self._args = []
        for c in calls:
            if c.x.shape[1] != c.k or c.y.shape != (c.x.shape[0], c.n):
                raise ValueError("inconsistent GEMV shapes")
            xt = W4_F32 if c.x.dtype == torch.float32 else W4_BF16
            yt = W4_F32 if c.y.dtype == torch.float32 else W4_BF16
            head = (ctypes.c_void_p(c.prepared.data_ptr()), c.n, c.k)
            tail = (ctypes.c_void_p(c.x.data_ptr()), xt, c.x.shape[0],
                    ctypes.c_void_p(c.y.data_ptr()), yt)
            if c.fmt is None:
                self._args.append((L.w4_gemv, "w4_gemv", head + tail))
            else:
                self._args.append((L.w4_gemv_fmt, "w4_gemv_fmt", head + (ctypes.byref(c.fmt),) + tail))

    def algorithmic_bytes(self) -> int:
        return sum(c.algorithmic_bytes() for c in self.calls)

    def run_eager(self) -> None:
        import torch
        s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        for fn, name, a in self._args:
            st = fn(*a, s)
            if st != 0:
                raise W4Error(st, name)

    def capture(self) -> None:
        """Record the whole step once into a graph (replayed by run())."""
        import torch
        self.run_eager()                      # warm caches and the device check outside capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run_eager()
        torch.cuda.synchronize()
        self._graph = g

    def run(self) -> None:
        if self._graph is not None:
            self._graph.replay()
        else:
            self.run_eager()


@dataclass
class Linear:
    """One product's weights: 4-bit (``prepared`` from w4_prepare), or FP8 / INT8 codes [N, K] (uint8 /
    int8 from w4_*_quantize_rows) with their row scales."""

    n: int
    k: int
    prepared: object = None
    codes: object = None
    scales: object = None

    @property
    def kind(self) -> str:
        if self.codes is None:
            return "w4"
        import torch
        return "fp8" if self.codes.dtype == torch.uint8 else "int8"


@dataclass
class DecoderLayer:
    """Norm weights [hidden] and the four products of a layer: q|k|v, attention output, gate|up, down."""

    attn_norm: object
    mlp_norm: object
    qkv: Linear
    o: Linear
    gate_up: Linear
    down: Linear


class DecoderStep:
    """Decoder layers over paged caches, for up to ``tokens`` new tokens of ``seqs`` requests a step.

    Before a step the caller writes the embeddings of the new tokens, request by request, into
    ``residual`` [tokens, hidden] and their number per request into ``new_lens`` [seqs]; the step places
    them in pages (``lens``, ``free_pages``, ``free_count`` and ``block_table`` go on from step to step,
    problems are reported in ``status``) and leaves the normed last hidden states in ``hidden``.
    Rows past the new tokens are padding; like the rows of requests that could not be served they are
    zeroed first (three small launches a step), so that nothing an earlier step left in them reaches the
    status.  4-bit products run on w4_gemv up to 16 tokens and on w4_gemm beyond; rows for 8-bit
    products are quantized by the operator that computes them.
    A request ends when the caller takes it out between two steps: with n the pages that its ``lens[b]``
    tokens fill, ``block_table[b, :n]`` goes to ``free_pages[free_count : free_count + n]``, ``free_count``
    grows by n and ``lens[b]`` becomes 0; the next request may then use its place.
    A step of another size over the same requests (a captured one for single tokens beside one for
    prompts) is made with ``state``, the step whose caches, lengths, pages, table and status it shares.
    ``tokens`` = ``seqs`` suits single tokens; a step that takes prompts should have another number of
    tokens, since the attention takes T = B for one token a request and is slower where it is not.
    """

    def __init__(self, layers, caches, heads, rope, final_norm, tokens, seqs, max_pages, eps=1e-5, free_pages=None,
                 state=None):
        import torch
        if not layers or len(layers) != len(caches):
            raise ValueError("one cache per layer")
        c = caches[0]
        if any((x.pages, x.page_size, x.kv_heads, x.head_dim) != (c.pages, c.page_size, c.kv_heads, c.head_dim) for x in caches):
            raise ValueError("the caches of all layers have one geometry")
        self.layers, self.caches, self.heads, self.rope, self.eps = layers, caches, heads, rope, eps
        self.final_norm, self.tokens, self.page_size = final_norm, tokens, c.page_size
        dev, hidden = c.device, layers[0].qkv.k
        self._device = dev
        width = (heads + 2 * c.kv_heads) * c.head_dim
        for a in layers:
            ffn = a.down.k
            want = ((a.qkv, width, hidden), (a.o, hidden, heads * c.head_dim), (a.gate_up, 2 * ffn, hidden), (a.down, hidden, ffn))
            if any((p.n, p.k) != (n, k) for p, n, k in want):
                raise ValueError("inconsistent layer shapes")
        i32, bf16 = dict(dtype=torch.int32, device=dev), dict(dtype=torch.bfloat16, device=dev)
        self.scale = c.head_dim ** -0.5
        self.freqs, _ = w4_rope_frequencies(rope, dev)
        self.residual, self.hidden = torch.zeros(tokens, hidden, **bf16), torch.zeros(tokens, hidden, **bf16)
        self.new_lens = torch.zeros(seqs, **i32)
        if state is not None:
            if (state.block_table.shape != (seqs, max_pages) or len(state.caches) != len(caches)
                    or any(x is not y for x, y in zip(state.caches, caches))):
                raise ValueError("state is of other requests")
            self.lens, self.free_pages, self.free_count = state.lens, state.free_pages, state.free_count
            self.block_table, self.status = state.block_table, state.status
        else:
            self.lens = torch.zeros(seqs, **i32)
            self.free_pages = torch.arange(c.pages, **i32) if free_pages is None else free_pages
            self.free_count = torch.full((1,), self.free_pages.numel(), **i32)
            self.block_table = torch.full((seqs, max_pages), -1, **i32)
            self.status = torch.zeros(1, **i32)
        self.cu_q, self.positions = torch.zeros(seqs + 1, **i32), torch.zeros(tokens, **i32)
        self.slots = torch.zeros(tokens, dtype=torch.int64, device=dev)
        self._x, self._y = torch.zeros(tokens, hidden, **bf16), torch.zeros(tokens, hidden, **bf16)
        self._qkv = torch.zeros(tokens, width, **bf16)
        self._qo = torch.zeros(2, tokens, heads, c.head_dim, **bf16)
        self._q, self._o = self._qo
        self._idle = torch.zeros(tokens, 1, dtype=torch.bool, device=dev)
        self._gate_up = {f: torch.zeros(tokens, 2 * f, **bf16) for f in {a.down.k for a in layers}}
        self._act = {f: torch.zeros(tokens, f, **bf16) for f in self._gate_up}
        products = [p for a in layers for p in (a.qkv, a.o, a.gate_up, a.down)]
        self._codes = {(p.kind, p.k): (torch.zeros(tokens, p.k, dtype=torch.uint8 if p.kind == "fp8" else torch.int8, device=dev),
                                       torch.zeros(tokens, dtype=torch.float32, device=dev)) for p in products if p.kind != "w4"}
        gemm = max([w4_gemm_workspace_bytes(tokens, p.n, p.k) for p in products if p.kind == "w4" and tokens > 16], default=0)
        self._gemm_workspace = torch.zeros(max(gemm, 16), dtype=torch.uint8, device=dev)
        from . import w4_paged_attention_workspace_bytes
        need = w4_paged_attention_workspace_bytes(tokens, heads, c, seqs, max_pages)
        self._attend_workspace = torch.zeros(max(need, 16), dtype=torch.uint8, device=dev)
        self._graph = None

    def _product(self, p, x, y):
        """y = x w^T; x: rows, or the codes and scales of rows."""
        if p.kind == "fp8":
            w4_fp8_gemm(x[0], x[1], p.codes, p.scales, Y=y)
        elif p.kind == "int8":
            w4_int8_gemm(x[0], x[1], p.codes, p.scales, Y=y)
        elif self.tokens <= 16:
            w4_gemv(p.prepared, p.n, p.k, x, y=y)
        else:
            w4_gemm(p.prepared, p.n, p.k, x, Y=y, workspace=self._gemm_workspace)

    def _norm(self, p, x, weight, residual):
        """Norm of the rows that feed product p, in the form that it takes."""
        from . import w4_rmsnorm, w4_rmsnorm_fp8, w4_rmsnorm_int8
        if p.kind == "w4":
            return w4_rmsnorm(x, weight, self.eps, residual=residual, y=self._x)
        codes, scales = self._codes[p.kind, p.k]
        call = w4_rmsnorm_fp8 if p.kind == "fp8" else w4_rmsnorm_int8
        return call(x, weight, self.eps, residual=residual, codes=codes, scales=scales, status=self.status)

    def _gate(self, p, gate_up):
        from . import w4_silu_mul, w4_silu_mul_fp8, w4_silu_mul_int8
        if p.kind == "w4":
            return w4_silu_mul(gate_up, y=self._act[p.k])
        codes, scales = self._codes[p.kind, p.k]
        call = w4_silu_mul_fp8 if p.kind == "fp8" else w4_silu_mul_int8
        return call(gate_up, codes=codes, scales=scales, status=self.status)

    def _rows(self, p, x):
        """Rows that are there as values, in the form that product p takes."""
        if p.kind == "w4":
            return x
        codes, scales = self._codes[p.kind, p.k]
        call = w4_fp8_quantize_rows if p.kind == "fp8" else w4_int8_quantize_rows
        return call(x, codes=codes, scales=scales, status=self.status)

    def run_eager(self) -> None:
        import torch
        with torch.cuda.device(self._device):                # some products launch on the current device
            self._step()

    def _step(self) -> None:
        import torch
        from . import w4_block_tables, w4_paged_attention, w4_rmsnorm, w4_rope_cache
        w4_block_tables(self.new_lens, self.lens, self.free_pages, self.free_count, self.block_table, self.page_size,
                        cu_q=self.cu_q, positions=self.positions, slots=self.slots, status=self.status)
        # Rows without a slot: the cache write and the attention leave them out, the products and norms do not.
        torch.lt(self.slots.view(-1, 1), 0, out=self._idle)
        self.residual.masked_fill_(self._idle, 0)
        self._qo.masked_fill_(self._idle.view(-1, 1, 1), 0)
        for i, (a, cache) in enumerate(zip(self.layers, self.caches)):
            if i == 0:
                x = self._norm(a.qkv, self.residual, a.attn_norm, None)
            else:
                x = self._norm(a.qkv, self._y, a.attn_norm, self.residual)
            self._product(a.qkv, x, self._qkv)
            w4_rope_cache(self._qkv, cache, self.positions, self.slots, self.rope, self.freqs, q=self._q, status=self.status)
            w4_paged_attention(self._q, cache, self.block_table, self.cu_q, self.lens, self.scale, o=self._o,
                               workspace=self._attend_workspace, status=self.status)
            self._product(a.o, self._rows(a.o, self._o.view(self.tokens, -1)), self._y)
            x = self._norm(a.gate_up, self._y, a.mlp_norm, self.residual)
            self._product(a.gate_up, x, self._gate_up[a.down.k])
            self._product(a.down, self._gate(a.down, self._gate_up[a.down.k]), self._y)
        w4_rmsnorm(self._y, self.final_norm, self.eps, residual=self.residual, y=self.hidden)

    def capture(self) -> None:
        """Record a step once into a graph (replayed by run()); what goes on from step to step, and
        ``residual``, is left as it was."""
        import torch
        with torch.cuda.device(self._device):
            kept = [t.clone() for t in self._state()]
            self.run_eager()                  # warm caches and the device check outside capture
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            # a stream of this device: the one that torch captures on by default stays on the first device used
            with torch.cuda.graph(g, stream=torch.cuda.Stream()):
                self.run_eager()
            for t, k in zip(self._state(), kept):
                t.copy_(k)
            torch.cuda.synchronize()
        self._graph = g

    def _state(self):
        return self.lens, self.free_count, self.block_table, self.status, self.residual

    def run(self) -> None:
        if self._graph is not None:
            self._graph.replay()
        else:
            self.run_eager()
