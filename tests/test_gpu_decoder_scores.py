"""DecoderStep over INT8 caches and with capped, biased or masked scores: prompts, then single tokens (eager and
captured), against a binary64 reference that goes through the same steps, writes the same blocks of its own INT8
caches and rounds where the path stores rows.

Tolerance as for the other caches (test_gpu_decoder_step): 2 * 4 * 2^-8 of the norm.  An INT8 code that lies on
either side of a rounding boundary for the two is off by a step, 1/127 of its block's largest value, about 2^-5 of
the values' root mean square; the attention averages such steps over its keys, so they stay below the half steps of
the four bfloat16 rows that the tolerance counts, as E4M3 rows with four times the step do there.
"""

import numpy as np
import pytest
import torch

import dequant_gemv_w4_amd as w4
import oracle
from dequant_gemv_w4_amd.decode import DecoderStep
from test_gpu_decoder_step import D, DEV, EPS, HEADS, HIDDEN, KV, TOL, Model, _check

pytestmark = pytest.mark.gpu


class Reference:
    """Steps of one request through the model's layers, with caches of its own."""

    def __init__(self, model, int8, rope, given, places):
        self.m, self.int8, self.rope, self.given = model, int8, rope, given
        self.n = 0
        pages = -(-places // 16)
        self.codes = [{n: np.zeros((pages, KV, 16, D), np.int8) for n in "kv"} for _ in model.ref]
        self.scales = [{n: np.zeros((pages, KV, 1), np.float32) for n in "kv"} for _ in model.ref]
        self.rows = [{n: np.zeros((KV, places, D)) for n in "kv"} for _ in model.ref]

    def _cached(self, i, k, v, at):
        ctx = at + len(k)
        out = []
        for n, x in (("k", k), ("v", v)):
            if self.int8:
                oracle.write_rows_ref(self.codes[i][n], self.scales[i][n], x, np.arange(at, ctx))
                rows = oracle.block_values(self.codes[i][n], self.scales[i][n])
                out.append(rows.transpose(1, 0, 2, 3).reshape(KV, -1, D)[:, :ctx])
            else:
                self.rows[i][n][:, at:ctx] = oracle.bf16_round(x.astype(np.float32)).transpose(1, 0, 2)
                out.append(self.rows[i][n][:, :ctx])
        return out

    def step(self, emb, first=None, prefix=None):
        m, n, at = self.m, len(emb), self.n
        self.n += n
        freqs, amp = oracle.rope_frequencies_ref(48, 10000.0, "linear", 2.0)
        r, y = emb, None
        for i, (norms, ref) in enumerate(m.ref):
            r = r if y is None else oracle.residual_sum_ref(y, r, True)
            qkv = m._product(ref["qkv"], oracle.rmsnorm_ref(r, norms[0], EPS)).reshape(n, HEADS + 2 * KV, D)
            qk = qkv[:, : HEADS + KV]
            if self.rope:
                qk = oracle.rope_ref(qk, np.arange(at, at + n), freqs, amp, m.interleaved).astype(np.float32)
            k, v = self._cached(i, qk[:, HEADS:], qkv[:, HEADS + KV:], at)
            o, _ = oracle.attention_scores_ref(oracle.bf16_round(qk[:, :HEADS]), k, v, at + n, D ** -0.5, first=first, prefix=prefix, **self.given)
            y = m._product(ref["o"], oracle.bf16_round(o.astype(np.float32)).reshape(n, -1))
            r = oracle.residual_sum_ref(y, r, True)
            y = m._product(ref["down"], oracle.silu_mul_ref(m._product(ref["gate_up"], oracle.rmsnorm_ref(r, norms[1], EPS))))
        return oracle.rmsnorm_ref(oracle.residual_sum_ref(y, r, True), m.final, EPS)


SLOPES = (0.5 ** np.arange(1, HEADS + 1)).astype(np.float32)


@pytest.mark.parametrize("int8,rope,given,ranges", [
    (True, True, {}, False), (True, False, dict(slopes=SLOPES), False), (False, True, dict(cap=3.0), False),
    (True, True, dict(cap=2.0), True), (False, False, dict(slopes=SLOPES, cap=5.0), True)])
def test_prompts_then_tokens(int8, rope, given, ranges):
    print(int8, rope, given, ranges, flush=True)
    m = Model(("w4",) * 4, False, 16, False, seed=41)
    g = np.random.default_rng(17)
    seqs, prefix = 3, np.array([9, 0, 30], np.int32)
    caches = [w4.W4KVCache.empty(40, 16, KV, D, device=DEV, int8=int8) for _ in m.layers]
    order = torch.from_numpy(g.permutation(40).astype(np.int32)).to(DEV)

    def made(tokens, state=None):
        kw = dict(given)
        if "slopes" in kw:
            kw["slopes"] = torch.from_numpy(kw["slopes"]).to(DEV)
        if ranges:
            kw.update(first_keys=torch.zeros(tokens, dtype=torch.int32, device=DEV), prefix_lens=torch.from_numpy(prefix).to(DEV))
        scores = w4.W4Scores(**kw) if kw else None
        return DecoderStep(m.layers, caches, HEADS, m.spec if rope else None, m.final_dev, tokens, seqs, 8, EPS,
                           free_pages=None if state else order, state=state, scores=scores)

    big = made(64)
    one = made(4, big)
    refs = [Reference(m, int8, rope, given, 128) for _ in range(seqs)]

    def step(s, new):
        emb = [oracle.bf16_round(g.standard_normal((n, HIDDEN)).astype(np.float32)) for n in new]
        rows = np.concatenate(emb)
        s.new_lens.copy_(torch.tensor(new, dtype=torch.int32))
        s.residual.zero_()
        s.residual[: len(rows)] = torch.from_numpy(rows).to(DEV).to(torch.bfloat16)
        firsts = [None] * seqs
        if ranges:                                            # documents of 25 tokens
            firsts = [(np.arange(r.n, r.n + n) // 25 * 25).astype(np.int32) for r, n in zip(refs, new)]
            s.scores[0].first_keys[: len(rows)] = torch.from_numpy(np.concatenate(firsts)).to(DEV)
        s.run()
        torch.cuda.synchronize()
        at = 0
        for b, n in enumerate(new):
            if n:
                want = refs[b].step(emb[b], firsts[b], int(prefix[b]) if ranges else None)
                _check(s.hidden[at: at + n], want, f"request {b}, {n} tokens up to {refs[b].n}", TOL)
            at += n
        assert s.lens.cpu().tolist() == [r.n for r in refs] and int(s.status) == 0

    step(big, [37, 1, 20])
    step(big, [0, 18, 40])
    step(one, [1, 1, 1])
    one.capture()
    for _ in range(4):
        step(one, [1, 0, 1])
    step(one, [1, 1, 2])
    big.capture()
    step(big, [15, 0, 5])
    step(one, [1, 0, 1])


def test_capture_leaves_an_int8_cache_as_it_was():
    m = Model(("w4",) * 4, False, 16, False, seed=43)
    caches = [w4.W4KVCache.empty(8, 16, KV, D, device=DEV, int8=True) for _ in m.layers]
    s = DecoderStep(m.layers, caches, HEADS, m.spec, m.final_dev, 8, 2, 4, EPS)
    s.new_lens.copy_(torch.tensor([3, 5], dtype=torch.int32))
    s.residual.copy_(torch.randn(8, HIDDEN, generator=torch.Generator().manual_seed(3)))
    s.run()
    torch.cuda.synchronize()
    before = [x.clone() for c in caches for x in (c.k, c.v, c.k_scales, c.v_scales)]
    s.residual.mul_(100.0)
    s.new_lens.fill_(1)
    kept = s.residual.clone()
    s.capture()
    assert all(torch.equal(x, y) for x, y in zip(before, [x for c in caches for x in (c.k, c.v, c.k_scales, c.v_scales)]))
    assert s.lens.cpu().tolist() == [3, 5] and s.new_lens.cpu().tolist() == [1, 1] and torch.equal(s.residual, kept)


def test_refusals():
    m = Model(("w4",) * 4, False, 16, False, seed=8)
    caches = [w4.W4KVCache.empty(4, 16, KV, D, device=DEV) for _ in m.layers]
    i32 = dict(dtype=torch.int32, device=DEV)
    for bad in ([None], w4.W4Scores(slopes=torch.zeros(HEADS + 1, device=DEV)), w4.W4Scores(first_keys=torch.zeros(5, **i32)),
                [None, w4.W4Scores(prefix_lens=torch.zeros(3, **i32))]):
        with pytest.raises(ValueError):
            DecoderStep(m.layers, caches, HEADS, m.spec, m.final_dev, 4, 2, 2, scores=bad)
    s = DecoderStep(m.layers, caches, HEADS, None, m.final_dev, 4, 2, 2, scores=[w4.W4Scores(cap=2.0), None])   # a record for each
    s.new_lens.copy_(torch.tensor([2, 1], dtype=torch.int32))
    s.run()
    torch.cuda.synchronize()
    assert int(s.status) == 0
