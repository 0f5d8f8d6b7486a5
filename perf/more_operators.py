"""Cases of the 8-bit cache with a scale for each block of tokens, and of attention whose scores or keys
are not the plain causal ones.

Four operators: the write of K and V into an INT8 cache with one scale per 16 tokens and head, with and
without rotary positions (`w4_rope_cache`, `w4_cache_write`), its rows read back as values
(`w4_cache_read`), attention over it (`w4_paged_attention`), and attention with capped scores, a bias by
distance, a document mask or a prefix mask (`w4_paged_attention_scores`).  With `own` false a pass runs
their plain form in elementary torch operations, with `own` true the framework's calls.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
INT8_MAX = 127.0
BLOCK = 16  # tokens that share a scale

# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------


def listed():
    return [
        # one decode step of a serving batch: a token of every request joins a block that is partly filled
        dict(name="write decode", op="write", seqs=64, new=1, cached=4000, heads=64, kv=8, d=128, rot=128, inter=False,
             page=16, x="f32"),
        # two prompts that go on behind cached tokens, of a model without rotary positions
        dict(name="write prompts", op="write", seqs=2, new=2048, cached=100, heads=32, kv=32, d=128, rot=0, inter=False,
             page=64, x="bf16"),
        # a short prefix of a request read back: latency
        dict(name="read short", op="read", n=129, kv=8, d=128, page=16, cache="int8", out="bf16"),
        # a long request's rows read back, to be moved or to be written into another cache
        dict(name="read long", op="read", n=65536, kv=8, d=128, page=64, cache="int8", out="bf16"),
        # one request's next token over a short context: latency
        _attend("int8 one token", seqs=1, new=1, cached=1000, heads=32, kv=8, d=64, page=16, cache="int8"),
        # a serving batch's decode step with ragged contexts
        _attend("int8 decode", seqs=32, new=1, cached=8192, heads=64, kv=8, d=128, page=16, cache="int8"),
        # chunks of prompts over what is cached of them
        _attend("int8 chunk", seqs=2, new=2048, cached=6144, heads=64, kv=8, d=128, page=32, cache="int8"),
        # a decode step of a model that caps its scores, in a layer with a window
        _attend("capped decode", seqs=16, new=1, cached=8192, heads=32, kv=16, d=128, page=32, cache="bf16", window=4096,
                cap=50.0, q=3.0),
        # a decode step of a model that knows positions by a bias alone, one kv head for each head
        _attend("bias decode", seqs=8, new=1, cached=16384, heads=32, kv=32, d=128, page=64, cache="int8", slopes=True),
        # short documents packed into one long prompt
        _attend("documents prompt", seqs=1, new=8192, cached=0, heads=32, kv=8, d=128, page=64, cache="bf16", docs=700),
        # prompts that begin with an image or an instruction whose tokens see each other
        _attend("prefix prompts", seqs=12, new=333, cached=50, heads=16, kv=2, d=64, page=16, cache="fp8", prefix=256, cap=30.0),
        # chunks of prompts of a model that caps its scores
        _attend("capped chunk", seqs=2, new=2048, cached=6144, heads=64, kv=8, d=128, page=32, cache="bf16", cap=50.0, q=3.0),
    ]


def _attend(name=None, **kw):
    """An attention case: what it does not say is off."""
    case = dict(op="attend", window=0, cap=0.0, slopes=False, docs=0, prefix=0, q=1.0)
    if name:
        case["name"] = name
    case.update(kw)
    return case


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("write", "read", "int8", "scores", "scores"))
    d = rng.choice((64, 128))
    page = 2 ** rng.randint(4, 8)
    if op == "read":
        kv = _log(rng, 1, 32)
        return dict(op=op, n=_log(rng, 1, 65536 * 8 // max(8, kv)), kv=kv, d=d, page=page,
                    cache=rng.choice(("int8", "int8", "bf16", "fp8")), out=rng.choice(("bf16", "f32")))
    kv, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 8))
    new = rng.choice((1, 1, _log(rng, 2, 16), _log(rng, 17, 1024)))
    if op == "write":
        return dict(op=op, seqs=_log(rng, 1, max(1, min(256, 4096 // new))), new=new, cached=_log(rng, 1, 100000) - 1,
                    heads=kv * group, kv=kv, d=d, rot=rng.choice((0, 16 * rng.randint(1, d // 16))), inter=rng.random() < 0.5,
                    page=page, x=rng.choice(("bf16", "f32")))
    cached = _log(rng, 1, 16384)
    # scores of the plain form no larger than half of the largest's, and caches no larger than its largest
    most = max(1, int(2048 * 8192 * 64 // (new * (new + cached) * kv * group)))
    room = max(1, int(2 ** 28 // ((new + cached) * kv * d)))
    case = _attend(seqs=_log(rng, 1, max(1, min(64, most, room))), new=new, cached=cached, heads=kv * group, kv=kv, d=d, page=page,
                   cache="int8" if op == "int8" else rng.choice(("bf16", "fp8", "int8")), window=rng.choice((0, 0, _log(rng, 1, 4096))))
    if op == "scores":
        form = rng.choice(("cap", "slopes", "docs", "prefix", "both"))
        if form in ("cap", "both"):
            case.update(cap=round(math.exp(rng.uniform(math.log(2.0), math.log(200.0))), 2), q=rng.choice((1.0, 3.0, 8.0)))
        if form in ("slopes", "both"):
            case["slopes"] = True
        if form == "docs" or rng.random() < 0.2:
            case["docs"] = _log(rng, 1, 4096)
        if form == "prefix" or rng.random() < 0.2:
            case["prefix"] = _log(rng, 1, new + cached)
    return case


def _lengths(case):
    """New and cached tokens of each request: the first has the most of both, the others are spread below."""
    n = case["seqs"]
    r = random.Random("%d %d %d" % (n, case["new"], case["cached"]))
    new = [case["new"]] + [r.randint(1, case["new"]) for _ in range(n - 1)]
    cached = [case["cached"]] + [r.randint(case["cached"] // 2, case["cached"]) for _ in range(n - 1)]
    return new, cached


def _prefixes(case):
    """Tokens at the start of each request that all of its rows see."""
    r = random.Random("%d %d" % (case["seqs"], case["prefix"]))
    return [r.randint(case["prefix"] // 2, case["prefix"]) for _ in range(case["seqs"])]


def _documents(case):
    """First key of each new token's document, as numpy arrays, request by request."""
    r = random.Random("%d %d %d" % (case["seqs"], case["new"], case["docs"]))
    out = []
    for n, c in zip(*_lengths(case)):
        starts = [0]
        while starts[-1] < n + c:
            starts.append(starts[-1] + r.randint(1, 2 * case["docs"]))
        starts = np.array(starts)
        pos = np.arange(c, c + n)
        out.append(starts[np.searchsorted(starts, pos, side="right") - 1])
    return out


def _visible(case):
    """Pairs of a query and a key that it sees, and keys that any query of their request sees."""
    new, cached = _lengths(case)
    docs = _documents(case) if case["docs"] else None
    prefix = _prefixes(case) if case["prefix"] else None
    pairs = keys = 0
    for b, (n, c) in enumerate(zip(new, cached)):
        pos = np.arange(c, c + n)
        lo, hi = np.zeros_like(pos), pos
        if case["window"]:
            lo = np.maximum(lo, pos - case["window"] + 1)
        if docs:
            lo = np.maximum(lo, docs[b])
        if prefix:
            hi = np.maximum(hi, min(prefix[b], n + c) - 1)
        pairs += int((hi - lo + 1).sum())
        edge = np.zeros(n + c + 1, dtype=np.int64)
        np.add.at(edge, lo, 1)
        np.add.at(edge, hi + 1, -1)
        keys += int((np.cumsum(edge) > 0).sum())
    return pairs, keys


SIZE = {"f32": 4, "bf16": 2, "fp8": 1, "int8": 1}


def _row_bytes(cache, d):
    """A cached row of one head with its share of the scales."""
    return d * SIZE[cache] + {"bf16": 0, "fp8": 4, "int8": 4 / BLOCK}[cache]


def work(case):
    op, d, kv = case["op"], case["d"], case["kv"]
    if op == "read":
        return {"bytes": int(case["n"] * (2 * kv * (_row_bytes(case["cache"], d) + d * SIZE[case["out"]]) + 8)), "flops": 2 * case["n"] * kv * d}
    new, cached = _lengths(case)
    t = sum(new)
    if op == "write":
        blocks = sum((n + c + BLOCK - 1) // BLOCK - c // BLOCK for n, c in zip(new, cached))
        return {"bytes": t * ((case["heads"] + 2 * kv) * d * SIZE[case["x"]] + case["heads"] * d * 2 + 2 * kv * d + 12) + blocks * 2 * kv * 8
                + 4 * case["rot"], "flops": t * ((case["heads"] + kv) * case["rot"] * 3 + 4 * kv * d)}
    pairs, keys = _visible(case)
    return {"bytes": int(keys * kv * 2 * _row_bytes(case["cache"], d)) + 2 * t * case["heads"] * d * 2, "flops": 4 * pairs * case["heads"] * d}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

TYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _rows(g, rows, k, dtype, large=20.0):
    """Activation rows: normal values, one channel in a hundred so many times as large."""
    x = torch.randn(rows, k, device=DEV, generator=g)
    big = torch.rand(k, device=DEV, generator=g) < 0.01
    x *= torch.where(big, large, 1.0)
    return x.to(dtype)


def _cache(case, pages, g):
    """A paged cache [pages, kv heads, page, d] filled with normal rows."""
    shape = (pages, case["kv"], case["page"], case["d"])
    got = {}
    for n in ("k", "v"):
        x = torch.randn(shape, device=DEV, generator=g, dtype=torch.bfloat16)
        got[n], got[n + "_scales"] = x, None
        if case["cache"] == "fp8":
            s = x.abs().amax(-1, keepdim=True).float() / E4M3_MAX
            got[n] = (x.float() / s).to(torch.float8_e4m3fn).view(torch.uint8)
            got[n + "_scales"] = s.squeeze(-1)
        if case["cache"] == "int8":
            blocks = x.view(*shape[:2], -1, BLOCK, shape[3])
            s = blocks.abs().amax((-1, -2)).float() / INT8_MAX
            got[n] = (blocks.float() / s[..., None, None]).round().to(torch.int8).view(shape)
            got[n + "_scales"] = s
    return got


def _frequencies(rot, base=500000.0):
    return [base ** (-2 * i / rot) for i in range(rot // 2)]


def _paged(case, g):
    """Block tables over shuffled pages for the requests' cached and new tokens."""
    new, cached = _lengths(case)
    p = case["page"]
    total = [n + c for n, c in zip(new, cached)]
    need = [(t + p - 1) // p for t in total]
    pages = sum(need) + 3
    order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
    at = torch.arange(max(need), device=DEV)
    start = torch.tensor([sum(need[:b]) for b in range(len(need))], device=DEV)
    used = at < torch.tensor(need, device=DEV)[:, None]
    table = torch.where(used, order[(start[:, None] + at).clamp_max(pages - 1)], -1).to(torch.int32)
    cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device=DEV)
    return dict(table=table.contiguous(), cu=cu, lens=torch.tensor(total, dtype=torch.int32, device=DEV), pages=pages,
                tokens=sum(new), most=max(new), longest=max(total))


def _write_state(case, g):
    """Rows of the fused q|k|v product, their positions and slots, and the pages that they go to.  What these pages hold
    was written like the new rows, so that some of the blocks that go on need a larger scale and most do not."""
    new, cached = _lengths(case)
    p, kv, d = case["page"], case["kv"], case["d"]
    ends = [c + n for n, c in zip(new, cached)]
    held = [(e + p - 1) // p - c // p for e, c in zip(ends, cached)]
    pages = sum(held) + 2
    order = torch.randperm(pages, generator=g, device=DEV)
    at, places, positions = 0, [], []
    for n, c, h in zip(new, cached, held):
        pos = np.arange(c, c + n)
        places.append(at + pos // p - c // p)
        positions.append(pos)
        at += h
    positions = torch.from_numpy(np.concatenate(positions)).to(DEV)
    places = torch.from_numpy(np.concatenate(places)).to(DEV)
    x = _rows(g, sum(new), (case["heads"] + 2 * kv) * d, TYPE[case["x"]])
    cache = {}
    for i, n in enumerate(("k", "v")):
        # the largest of what these heads' rows hold, a little less or more
        most = x.view(len(x), -1, d)[:, case["heads"] + i * kv: case["heads"] + (i + 1) * kv].abs().amax((0, 2)).float()
        cache[n] = (40 * torch.randn(pages, kv, p, d, device=DEV, generator=g)).clamp_(-INT8_MAX, INT8_MAX).round_().to(torch.int8)
        cache[n + "_scales"] = (most[:, None] / INT8_MAX * (0.5 + 0.6 * torch.rand(pages, kv, p // BLOCK, device=DEV, generator=g))).contiguous()
    s = dict(case=case, cache=cache, x=x, positions=positions.to(torch.int32), slots=(order[places] * p + positions % p).contiguous(),
             q=torch.empty(sum(new), case["heads"], d, dtype=torch.bfloat16, device=DEV))
    if case["rot"]:
        s["freqs"] = torch.tensor(_frequencies(case["rot"]), dtype=torch.float64, device=DEV)
    if own:
        import dequant_gemv_w4_amd as w4
        s["kv"] = w4.W4KVCache(**cache)
        if case["rot"]:
            s["rope"] = w4.W4Rope.make(case["rot"], base=500000.0, interleaved=case["inter"])
    return s


def _read_state(case, g):
    """The slots of a request's tokens in shuffled pages, one token short of a page's end where there are several."""
    p, n = case["page"], case["n"]
    pages = (n + p - 1) // p + 1
    order = torch.randperm(pages, generator=g, device=DEV)
    pos = torch.arange(n, device=DEV)
    cache = _cache(case, pages, g)
    s = dict(case=case, cache=cache, slots=(order[pos // p] * p + pos % p).contiguous(),
             out=torch.empty(n, 2 * case["kv"] * case["d"], dtype=TYPE[case["out"]], device=DEV))
    if own:
        import dequant_gemv_w4_amd as w4
        s["kv"] = w4.W4KVCache(**cache)
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] == "write":
        return _write_state(case, g)
    if case["op"] == "read":
        return _read_state(case, g)
    s = _paged(case, g)
    cache = _cache(case, s["pages"], g)
    shape = (s["tokens"], case["heads"], case["d"])
    s.update(case=case, cache=cache, scale=case["d"] ** -0.5,
             q=(case["q"] * torch.randn(shape, device=DEV, generator=g)).bfloat16(),
             o=torch.empty(shape, dtype=torch.bfloat16, device=DEV), slopes=None, first=None, prefix=None)
    if case["slopes"]:  # powers of one ratio, as models that know positions by a bias take them
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, case["heads"] + 1, dtype=torch.float32, device=DEV) / case["heads"])
    if case["docs"]:
        s["first"] = torch.from_numpy(np.concatenate(_documents(case))).to(DEV).to(torch.int32)
    if case["prefix"]:
        s["prefix"] = torch.tensor(_prefixes(case), dtype=torch.int32, device=DEV)
    if own:
        import dequant_gemv_w4_amd as w4
        s["kv"] = w4.W4KVCache(**cache)
        s["workspace"] = torch.empty(max(1, w4.w4_paged_attention_workspace_bytes(
            s["q"].shape[0], case["heads"], s["kv"], case["seqs"], s["table"].shape[1])), dtype=torch.uint8, device=DEV)
        if case["cap"] or case["slopes"] or case["docs"] or case["prefix"]:
            s["scores"] = w4.W4Scores(cap=case["cap"], slopes=s["slopes"], first_keys=s["first"], prefix_lens=s["prefix"])
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------


def run(state):
    return (_run_own if own else _run_plain)(state)


def _cache_out(q, c):
    """q and the cache: codes as the whole numbers that they are, in bf16 (which holds them), and the scales."""
    return [q, c["k"].to(torch.bfloat16), c["v"].to(torch.bfloat16), c["k_scales"], c["v_scales"]]


def _run_own(s):
    import dequant_gemv_w4_amd as w4
    case = s["case"]
    if case["op"] == "write":
        if case["rot"]:
            w4.w4_rope_cache(s["x"], s["kv"], s["positions"], s["slots"], s["rope"], s["freqs"], q=s["q"])
        else:
            w4.w4_cache_write(s["x"], s["kv"], s["slots"], q=s["q"])
        return _cache_out(s["q"], s["cache"])
    if case["op"] == "read":
        return [w4.w4_cache_read(s["kv"], s["slots"], out=s["out"])]
    kept = dict(window=case["window"], o=s["o"], workspace=s["workspace"])
    if "scores" in s:
        return [w4.w4_paged_attention_scores(s["q"], s["kv"], s["table"], s["cu"], s["lens"], s["scale"], s["scores"], **kept)]
    return [w4.w4_paged_attention(s["q"], s["kv"], s["table"], s["cu"], s["lens"], s["scale"], **kept)]


def _run_plain(s):
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[s["case"]["op"]](s)


def _plain_write(s):
    case = s["case"]
    h, kv, d, half, p = case["heads"], case["kv"], case["d"], case["rot"] // 2, case["page"]
    y = s["x"].float().view(-1, h + 2 * kv, d)
    if half:
        a = s["positions"].double()[:, None] * s["freqs"]
        cos, sin = (f(a).float()[:, None] for f in (torch.cos, torch.sin))
        x, y = y, y.clone()
        if case["inter"]:
            first, second = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
        else:
            first, second = slice(0, half), slice(half, 2 * half)
        x0, x1 = x[:, : h + kv, first], x[:, : h + kv, second]
        y[:, : h + kv, first], y[:, : h + kv, second] = x0 * cos - x1 * sin, x0 * sin + x1 * cos
    page, at = s["slots"] // p, s["slots"] % p
    for n, rows in (("k", y[:, h: h + kv]), ("v", y[:, h + kv:])):
        codes, scales = s["cache"][n], s["cache"][n + "_scales"]
        pages = codes.shape[0]
        block = page * (p // BLOCK) + at // BLOCK
        by_block = scales.transpose(1, 2).reshape(-1, kv)
        # blocks whose first row is written begin anew
        starts = torch.zeros(by_block.shape[0], device=DEV).index_add_(0, block, (at % BLOCK == 0).float()) > 0
        old = torch.where(starts[:, None], 0.0, by_block)
        need = torch.zeros_like(by_block).scatter_reduce_(0, block[:, None].expand(-1, kv), rows.abs().amax(-1) / INT8_MAX, "amax")
        touched = torch.zeros_like(starts)
        touched[block] = True
        new = torch.where(touched[:, None], torch.maximum(old, need), by_block)
        keep = torch.where(touched[:, None] & ~starts[:, None] & (new > old), old / new, 1.0)

        def spread(t):  # [blocks, kv] -> [pages, kv, rows of a page, 1]
            return t.view(pages, -1, kv).transpose(1, 2).repeat_interleave(BLOCK, 2).unsqueeze(-1)

        codes.copy_((codes.float() * spread(keep)).round())
        codes[page, :, at] = (rows / new[block][..., None]).round().to(torch.int8)
        scales.copy_(new.view(pages, -1, kv).transpose(1, 2))
    return _cache_out(y[:, :h].bfloat16(), s["cache"])


def _values(c, n, page, at, dtype):
    """Rows [..., kv heads, d] of a cache by pages and places in them."""
    x = c[n][page, :, at]
    if x.dtype == torch.bfloat16:
        return x.to(dtype)
    if x.dtype == torch.uint8:
        return x.view(torch.float8_e4m3fn).to(dtype) * c[n + "_scales"][page, :, at].to(dtype)[..., None]
    return x.to(dtype) * c[n + "_scales"][page, :, at // BLOCK].to(dtype)[..., None]


def _plain_read(s):
    p = s["case"]["page"]
    page, at = s["slots"] // p, s["slots"] % p
    both = [_values(s["cache"], n, page, at, torch.float32) for n in ("k", "v")]
    return [torch.cat(both, 1).flatten(1).to(s["out"].dtype)]


def _plain_attend(s):
    case = s["case"]
    n, p, h, kv, d = case["seqs"], case["page"], case["heads"], case["kv"], case["d"]
    most, longest = s["most"], s["longest"]
    j = torch.arange(longest, device=DEV)
    page = s["table"].long()[:, j // p].clamp_min(0)
    k, v = (_values(s["cache"], x, page, (j % p).expand_as(page), torch.float32).transpose(1, 2).contiguous() for x in ("k", "v"))
    cu, lens = s["cu"].long(), s["lens"].long()
    i = torch.arange(most, device=DEV)
    real = i < (cu[1:] - cu[:-1])[:, None]
    rows = torch.where(real, cu[:-1, None] + i, 0)
    q = s["q"][rows].float().view(n, most, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(n, kv, -1, d)
    z = torch.matmul(q, k.transpose(-1, -2).contiguous()).view(n, h, most, longest).mul_(s["scale"])
    if case["cap"]:
        z = z.div_(case["cap"]).tanh_().mul_(case["cap"])
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + i
    if s["slopes"] is not None:
        away = (pos[..., None] - j).abs().float()
        z.addcmul_(s["slopes"][:, None, None], away[:, None], value=-1.0)
    last = pos
    if s["prefix"] is not None:
        last = torch.maximum(pos, s["prefix"].long()[:, None] - 1)
    seen = (j <= last[..., None]) & (j < lens[:, None, None])
    if case["window"]:
        seen &= j > pos[..., None] - case["window"]
    if s["first"] is not None:
        seen &= j >= s["first"].long()[rows][..., None]
    z.masked_fill_(~seen[:, None], -math.inf)
    z = z.sub_(z.amax(-1, keepdim=True).clamp_min(-3e38)).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(n, kv, -1, longest), v).view(n, h, most, d) / total
    return [o.transpose(1, 2)[real].bfloat16()]


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attend": _exact_attend}[case["op"]](case, s)


def _exact_write(case, s):
    h, kv, d, rot, p = case["heads"], case["kv"], case["d"], case["rot"], case["page"]
    x = s["x"].double().view(-1, h + 2 * kv, d).clone()
    if rot:
        z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), torch.outer(s["positions"].double(), s["freqs"]))
        part = x[:, : h + kv, :rot]
        part = part.unflatten(-1, (-1, 2)) if case["inter"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
        turned = torch.view_as_real(torch.view_as_complex(part.contiguous()) * z[:, None])
        x[:, : h + kv, :rot] = (turned if case["inter"] else turned.transpose(-1, -2)).flatten(-2)
    out, scales = [x[:, :h]], []
    # the tokens of each block that the write touches, one block after the other, all heads at once
    slots = s["slots"].tolist()
    blocks = {}
    for t, slot in enumerate(slots):
        blocks.setdefault(slot // BLOCK, []).append(t)
    for first, n in ((h, "k"), (h + kv, "v")):
        codes = s["cache"][n].double().clone()
        steps = s["cache"][n + "_scales"].double().clone()
        for b, tokens in blocks.items():
            page, at = b * BLOCK // p, b * BLOCK % p
            rows = x[tokens, first: first + kv]
            where = [slots[t] % BLOCK for t in tokens]
            before = torch.zeros(kv, dtype=torch.float64, device=DEV) if 0 in where else steps[page, :, at // BLOCK].clone()
            after = torch.maximum(before, rows.abs().amax((0, 2)) / 127)
            if 0 not in where:
                held = codes[page, :, at: at + BLOCK]
                held *= (before / after)[:, None, None]
                held.round_()
            codes[page, :, [at + w for w in where]] = (rows / after[:, None]).round().transpose(0, 1)
            steps[page, :, at // BLOCK] = after
        out.append(codes)
        scales.append(steps)
    return out + scales


def _exact_read(case, s):
    p, kv, d = case["page"], case["kv"], case["d"]
    out = torch.empty(case["n"], 2, kv, d, dtype=torch.float64, device=DEV)
    for i, n in enumerate(("k", "v")):
        flat = s["cache"][n].transpose(1, 2).reshape(-1, kv, d)
        x = flat[s["slots"]]
        out[:, i] = x.view(torch.float8_e4m3fn).double() if case["cache"] == "fp8" else x.double()
        if case["cache"] != "bf16":
            per = s["cache"][n + "_scales"].transpose(1, 2).reshape(-1, kv).double()
            out[:, i] *= per[s["slots"] if case["cache"] == "fp8" else torch.div(s["slots"], BLOCK, rounding_mode="floor")][..., None]
    return [out.flatten(1)]


def _exact_attend(case, s):
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    group, p = case["heads"] // case["kv"], case["page"]
    for b in range(case["seqs"]):
        length, n = lens[b], cu[b + 1] - cu[b]
        j = torch.arange(length, device=DEV)
        pages = s["table"][b].long()[j // p]
        pos = torch.arange(length - n, length, device=DEV)[:, None]
        hidden = j > pos
        if s["prefix"] is not None:
            hidden &= j >= s["prefix"][b]
        if case["window"]:
            hidden |= j <= pos - case["window"]
        if s["first"] is not None:
            hidden |= j < s["first"][cu[b]: cu[b + 1], None]
        away = (pos - j).abs().double()
        for head in range(case["heads"]):
            k, v = (_one_head(s["cache"], x, pages, head // group, j % p) for x in ("k", "v"))
            z = (s["q"][cu[b]: cu[b + 1], head].double() @ k.t().contiguous()) * s["scale"]
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if s["slopes"] is not None:
                z = z - s["slopes"][head].double() * away
            out[cu[b]: cu[b + 1], head] = torch.softmax(z.masked_fill_(hidden, -math.inf), -1) @ v
    return [out]


def _one_head(c, n, pages, head, at):
    x = c[n][pages, head, at]
    if c[n + "_scales"] is None:
        return x.double()
    if x.dtype == torch.uint8:
        return x.view(torch.float8_e4m3fn).double() * c[n + "_scales"][pages, head, at].double()[:, None]
    return x.double() * c[n + "_scales"][pages, head, at // BLOCK].double()[:, None]
