"""DecoderStep at its edges: rows that become padding after they held a value that is not finite, and
requests that are refused; requests that end and give their pages back; a state whose caches are
others; a device that is not the current one."""

import numpy as np
import pytest
import torch

import dequant_gemv_w4_amd as w4
import oracle
from dequant_gemv_w4_amd.decode import DecoderStep
from test_gpu_decoder_step import D, DEV, EPS, HEADS, HIDDEN, KV, MORE, TOL, Model, _check

pytestmark = pytest.mark.gpu


def _put(s, new, rows):
    s.new_lens.copy_(torch.tensor(new, dtype=torch.int32))
    s.residual[: len(rows)] = rows


@pytest.mark.parametrize("kind", ["fp8", "int8", "w4"])
@pytest.mark.parametrize("fp8_cache", [False, True])
@pytest.mark.parametrize("capture", [False, True])
def test_rows_that_become_padding(kind, fp8_cache, capture):
    m = Model((kind,) * 4, fp8_cache, 16, False, seed=12)
    caches = [w4.W4KVCache.empty(12, 16, KV, D, fp8=fp8_cache, device=DEV) for _ in m.layers]
    s = DecoderStep(m.layers, caches, HEADS, m.spec, m.final_dev, 6, 4, 4, EPS)
    rows = torch.randn(6, HIDDEN, generator=torch.Generator().manual_seed(2)).to(DEV).to(torch.bfloat16)
    if capture:
        s.capture()
    bad = rows.clone()
    bad[3:] = float("nan")                                    # request 3's three tokens
    _put(s, [1, 1, 1, 3], bad)
    s.run()
    torch.cuda.synchronize()
    assert bool(torch.isfinite(s.hidden[:3].float()).all()) and not bool(torch.isfinite(s.hidden[3:].float()).any())
    assert int(s.status) == (0 if kind == "w4" and not fp8_cache else 1)
    s.status.zero_()
    _put(s, [1, 1, 1, 0], rows[:3])                           # the rows behind are padding now
    s.run()
    torch.cuda.synchronize()
    assert int(s.status) == 0 and bool(torch.isfinite(s.hidden[:3].float()).all())
    _put(s, [1, 9, 0, 0], rows)                               # and here those of a request that has too many tokens
    s.run()
    torch.cuda.synchronize()
    assert int(s.status) == 16 and bool(torch.isfinite(s.hidden[:1].float()).all())
    assert s.lens.cpu().tolist() == [3, 2, 2, 3]


@pytest.mark.parametrize("kind,fp8_cache", [("w4", False), ("fp8", True)])
def test_requests_end_and_others_take_their_pages(kind, fp8_cache):
    # the pages of the request that ends go back to the list behind the free ones; the next takes them
    page, pages, wide = 16, 6, 4
    m = Model((kind,) * 4, fp8_cache, page, False, seed=14)
    g = np.random.default_rng(3)
    caches = [w4.W4KVCache.empty(pages, page, KV, D, fp8=fp8_cache, device=DEV) for _ in m.layers]
    s = DecoderStep(m.layers, caches, HEADS, m.spec, m.final_dev, 64, 2, wide, EPS)
    tol = TOL + MORE[kind]
    other = oracle.bf16_round(g.standard_normal((4, HIDDEN)).astype(np.float32))
    other_ref = m.forward(other)
    done = 0
    for n in (50, 37, 60, 33):                                # 4 or 3 of 5 pages: none fits beside its predecessor
        emb = oracle.bf16_round(g.standard_normal((n, HIDDEN)).astype(np.float32))
        _put(s, [n, 1], torch.from_numpy(np.concatenate([emb, other[done: done + 1]])).to(DEV).to(torch.bfloat16))
        s.run()
        torch.cuda.synchronize()
        assert int(s.status) == 0 and s.lens.cpu().tolist() == [n, done + 1]
        _check(s.hidden[:n], m.forward(emb), f"request of {n} tokens", tol)
        _check(s.hidden[n: n + 1], other_ref[done: done + 1], f"token {done} beside it", tol)
        done += 1
        held, count = -(-n // page), int(s.free_count)
        s.free_pages[count: count + held] = s.block_table[0, :held]
        s.free_count += held
        s.block_table[0] = -1
        s.lens[0] = 0
        assert sorted(s.free_pages[: count + held].tolist() + s.block_table[1, :1].tolist()) == list(range(pages))


def test_state_of_other_caches_is_refused():
    m = Model(("w4",) * 4, False, 16, False, seed=8)
    caches = [w4.W4KVCache.empty(2, 16, KV, D, device=DEV) for _ in m.layers]
    s = DecoderStep(m.layers, caches, HEADS, m.spec, m.final_dev, 4, 1, 2)
    DecoderStep(m.layers, list(caches), HEADS, m.spec, m.final_dev, 2, 1, 2, state=s)
    others = [caches[0]] + [w4.W4KVCache.empty(2, 16, KV, D, device=DEV) for _ in m.layers[1:]]
    with pytest.raises(ValueError):
        DecoderStep(m.layers, others, HEADS, m.spec, m.final_dev, 2, 1, 2, state=s)


def test_capture_on_the_step_s_own_device(monkeypatch):
    # A graph records what goes to the capturing stream of one device: the step has to make its device the
    # current one and capture on a stream of it.  One GPU is here, so the calls that do it are watched.
    m = Model(("w4",) * 4, False, 16, False, seed=8)
    caches = [w4.W4KVCache.empty(2, 16, KV, D, device=DEV) for _ in m.layers]
    s = DecoderStep(m.layers, caches, HEADS, m.spec, m.final_dev, 4, 1, 2)
    inside, real_device, real_graph = [], torch.cuda.device, torch.cuda.graph
    graphs = []

    class Device(real_device):
        def __enter__(self):
            inside.append(self.idx)
            return super().__enter__()

        def __exit__(self, *a):
            inside.pop()
            return super().__exit__(*a)

    def graph(g, **kw):
        graphs.append((list(inside), kw["stream"].device.index if kw.get("stream") is not None else None))
        return real_graph(g, **kw)

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "graph", graph)
    s.capture()
    assert graphs == [([0], 0)]
    s.new_lens.fill_(2)
    s.run()
    torch.cuda.synchronize()
    assert s.lens.cpu().tolist() == [2] and int(s.status) == 0
