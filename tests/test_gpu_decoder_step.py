"""DecoderStep: whole decoder layers over paged caches, prompts first and then single tokens (eager
and captured), against a binary64 forward pass over each request's whole sequence that rounds where
the path stores bfloat16 or 8-bit rows.

Between equal rounding points the two differ by binary32 arithmetic (which now and then turns a
rounding), and by the attention's bfloat16 weights (half step 2^-8 each).  A layer has four stored
rows behind such a difference on the residual path (o, its product, gate, its product), so the last
hidden states of two layers may be off by 2 * 4 * 2^-8 of their norm at most; a wrong head, page,
position or order is off by about the norm itself.

8-bit rows turn such small differences into whole steps: a value that lies on either side of a
rounding boundary for the two gets neighbouring codes, and after a few rows most roundings are
independent of each other.  A rounding's error is then uniform within half a step, 2^-4 of the value for
E4M3 and 2^-8 of the row's largest value, about 4 times its root mean square, for INT8, so with
independent errors on both sides in the four stored rows of each of two layers the norms differ by
sqrt(2 * 8) * 2^-4 / sqrt(3) = 0.144 and sqrt(2 * 8) * 2^-6 / sqrt(3) = 0.036 more.
"""

import numpy as np
import pytest
import torch

import dequant_gemv_w4_amd as w4
import oracle
from dequant_gemv_w4_amd.decode import DecoderLayer, DecoderStep, Linear
from _util import to_np32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HIDDEN, HEADS, KV, D, FFN, EPS = 256, 4, 2, 64, 384, 1e-5
TOL = 2 * 4 * 2.0 ** -8
MORE = {"w4": 0.0, "fp8": 4 * 2.0 ** -4 / 3 ** 0.5, "int8": 4 * 2.0 ** -6 / 3 ** 0.5}


class Model:
    def __init__(self, kinds, fp8_cache, page, interleaved, seed):
        g = np.random.default_rng(seed)
        self.fp8_cache, self.interleaved = fp8_cache, interleaved
        self.spec = w4.W4Rope.make(48, 10000.0, interleaved, "linear", 2.0)
        self.layers, self.ref = [], []
        shapes = dict(qkv=((HEADS + 2 * KV) * D, HIDDEN), o=(HIDDEN, HEADS * D), gate_up=(2 * FFN, HIDDEN), down=(HIDDEN, FFN))
        for _ in range(2):
            made, ref = {}, {}
            for (name, (n, k)), kind in zip(shapes.items(), kinds):
                W = torch.from_numpy((g.standard_normal((n, k)) * k ** -0.5).astype(np.float32)).to(DEV)
                if kind == "w4":
                    p, s, z = w4.w4_quantize(W)
                    made[name] = Linear(n, k, prepared=w4.w4_prepare(p, s, z))
                    ref[name] = (kind, oracle.dequant_ref(p.cpu().numpy(), s.cpu().numpy(), z.cpu().numpy()).astype(np.float64))
                else:
                    c, s = (w4.w4_fp8_quantize_rows if kind == "fp8" else w4.w4_int8_quantize_rows)(W)
                    made[name] = Linear(n, k, codes=c, scales=s)
                    ref[name] = (kind, self._values(kind, c.cpu().numpy(), s.cpu().numpy()))
            norms = [oracle.bf16_round((1 + 0.1 * g.standard_normal(HIDDEN)).astype(np.float32)) for _ in range(2)]
            dev = [torch.from_numpy(x).to(DEV).to(torch.bfloat16) for x in norms]
            self.layers.append(DecoderLayer(dev[0], dev[1], **made))
            self.ref.append((norms, ref))
        self.final = oracle.bf16_round((1 + 0.1 * g.standard_normal(HIDDEN)).astype(np.float32))
        self.final_dev = torch.from_numpy(self.final).to(DEV).to(torch.bfloat16)
        self.page = page

    @staticmethod
    def _values(kind, codes, scales):
        return (oracle.dequant_fp8_ref if kind == "fp8" else oracle.dequant_int8_ref)(codes, scales).astype(np.float64)

    def _product(self, part, rows):
        """rows: binary32 values before they are stored for the product."""
        kind, W = part
        rows = rows.astype(np.float32)
        if kind == "w4":
            x = oracle.bf16_round(rows)
        else:
            x = self._values(kind, *(oracle.quantize_rows_fp8_ref if kind == "fp8" else oracle.quantize_rows_int8_ref)(rows))
        return oracle.bf16_round((x.astype(np.float64) @ W.T).astype(np.float32))

    def forward(self, emb):
        """emb [n, HIDDEN] of one request -> normed hidden states."""
        n = len(emb)
        freqs, amp = oracle.rope_frequencies_ref(48, 10000.0, "linear", 2.0)
        r, y = emb, None
        for norms, ref in self.ref:
            r = r if y is None else oracle.residual_sum_ref(y, r, True)
            qkv = self._product(ref["qkv"], oracle.rmsnorm_ref(r, norms[0], EPS)).reshape(n, HEADS + 2 * KV, D)
            turned = oracle.rope_ref(qkv[:, : HEADS + KV], np.arange(n), freqs, amp, self.interleaved).astype(np.float32)
            q, k, v = oracle.bf16_round(turned[:, :HEADS]), turned[:, HEADS:], qkv[:, HEADS + KV:]
            if self.fp8_cache:
                k, v = (self._values("fp8", *oracle.quantize_rows_fp8_ref(np.ascontiguousarray(t).reshape(-1, D))).reshape(n, KV, D) for t in (k, v))
            else:
                k = oracle.bf16_round(k)
            o, _ = oracle.attention_ref(q, k.transpose(1, 0, 2), v.transpose(1, 0, 2), n, D ** -0.5)
            o = oracle.bf16_round(o.astype(np.float32)).reshape(n, -1)
            y = self._product(ref["o"], o)
            r = oracle.residual_sum_ref(y, r, True)
            gate_up = self._product(ref["gate_up"], oracle.rmsnorm_ref(r, norms[1], EPS))
            y = self._product(ref["down"], oracle.silu_mul_ref(gate_up))
        return oracle.rmsnorm_ref(oracle.residual_sum_ref(y, r, True), self.final, EPS)


def _check(got, ref, what, tol):
    got = to_np32(got).astype(np.float64)
    off = np.linalg.norm(got - ref, axis=1) / np.linalg.norm(ref, axis=1)
    assert off.max() <= tol, f"{what}: off by {off.max():.4f} of the norm, {tol:.4f} allowed"


@pytest.mark.parametrize("kinds,fp8_cache,page,interleaved", [
    (("w4",) * 4, False, 16, False), (("w4",) * 4, True, 32, True), (("fp8",) * 4, True, 16, False),
    (("int8",) * 4, False, 64, True), (("w4", "fp8", "int8", "w4"), False, 16, False)])
def test_prompts_then_tokens(kinds, fp8_cache, page, interleaved):
    print(kinds, fp8_cache, flush=True)
    m = Model(kinds, fp8_cache, page, interleaved, seed=31)
    g = np.random.default_rng(7)
    seqs, total = 3, [60, 21, 75]
    emb = [oracle.bf16_round(g.standard_normal((n, HIDDEN)).astype(np.float32)) for n in total]
    want = [m.forward(e) for e in emb]
    caches = [w4.W4KVCache.empty(40, page, KV, D, fp8=fp8_cache, device=DEV) for _ in m.layers]
    order = torch.from_numpy(g.permutation(40).astype(np.int32)).to(DEV)
    big = DecoderStep(m.layers, caches, HEADS, m.spec, m.final_dev, 64, seqs, 8, EPS, free_pages=order)
    one = DecoderStep(m.layers, caches, HEADS, m.spec, m.final_dev, 4, seqs, 8, EPS, state=big)
    done = [0] * seqs
    tol = TOL + max(MORE[k] for k in kinds)

    def step(s, new):
        s.new_lens.copy_(torch.tensor(new, dtype=torch.int32))
        rows = np.concatenate([emb[b][done[b]: done[b] + n] for b, n in enumerate(new)])
        s.residual.zero_()
        s.residual[: len(rows)] = torch.from_numpy(rows).to(DEV).to(torch.bfloat16)
        s.run()
        torch.cuda.synchronize()
        at = 0
        for b, n in enumerate(new):
            if n:
                _check(s.hidden[at: at + n], want[b][done[b]: done[b] + n], f"request {b}, tokens {done[b]}..{done[b] + n}", tol)
            at += n
            done[b] += n
        assert s.lens.cpu().tolist() == done and int(s.status) == 0

    step(big, [37, 1, 20])                                    # prompts
    step(big, [0, 18, 40])                                    # the rest of a prompt beside nothing of another
    step(one, [1, 1, 1])
    one.capture()
    for _ in range(4):                                        # replays move on from where the last one left
        step(one, [1, 0, 1])
    step(one, [1, 1, 2])                                      # the same graph with other numbers
    big.capture()
    step(big, [15, 0, 5])
    step(one, [1, 0, 1])
    assert done == [37 + 1 + 4 + 1 + 15 + 1, 1 + 18 + 1 + 1, 20 + 40 + 1 + 4 + 2 + 5 + 1]
    assert int(one.free_count) == 40 - sum(-(-n // page) for n in done)


def test_captured_step_equals_eager_step():
    m = Model(("w4",) * 4, False, 16, False, seed=5)
    out = []
    for capture in (False, True):
        caches = [w4.W4KVCache.empty(12, 16, KV, D, device=DEV) for _ in m.layers]
        s = DecoderStep(m.layers, caches, HEADS, m.spec, m.final_dev, 8, 2, 4, EPS)
        s.new_lens.copy_(torch.tensor([2, 3], dtype=torch.int32))
        if capture:
            s.capture()
        got = []
        for i in range(5):
            s.residual.copy_(torch.randn(8, HIDDEN, generator=torch.Generator().manual_seed(i)))
            s.run()
            torch.cuda.synchronize()
            got.append((s.hidden[:5].clone(), s.lens.clone(), s.free_count.clone(), caches[1].k.clone()))
        out.append(got)
    for a, b in zip(*out):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_step_reports_and_survives_a_full_cache():
    m = Model(("w4",) * 4, False, 16, False, seed=6)
    caches = [w4.W4KVCache.empty(2, 16, KV, D, device=DEV) for _ in m.layers]
    s = DecoderStep(m.layers, caches, HEADS, m.spec, m.final_dev, 40, 2, 4, EPS)
    s.new_lens.copy_(torch.tensor([20, 17], dtype=torch.int32))
    s.residual.copy_(torch.randn(40, HIDDEN, generator=torch.Generator().manual_seed(1)))
    s.run()
    torch.cuda.synchronize()
    assert int(s.status) & 32 and s.lens.cpu().tolist() == [20, 0] and int(s.free_count) == 0
    assert bool(torch.isfinite(s.hidden[:20].float()).all())


def test_step_refusals():
    m = Model(("w4",) * 4, False, 16, False, seed=8)
    caches = [w4.W4KVCache.empty(2, 16, KV, D, device=DEV) for _ in m.layers]
    with pytest.raises(ValueError):
        DecoderStep(m.layers, caches[:1], HEADS, m.spec, m.final_dev, 4, 1, 2)
    with pytest.raises(ValueError):
        DecoderStep(m.layers, [caches[0], w4.W4KVCache.empty(3, 16, KV, D, device=DEV)], HEADS, m.spec, m.final_dev, 4, 1, 2)
    with pytest.raises(ValueError):
        DecoderStep(m.layers, caches, HEADS + 2, m.spec, m.final_dev, 4, 1, 2)
    s = DecoderStep(m.layers, caches, HEADS, m.spec, m.final_dev, 4, 1, 2)
    with pytest.raises(ValueError):
        DecoderStep(m.layers, caches, HEADS, m.spec, m.final_dev, 4, 2, 2, state=s)
