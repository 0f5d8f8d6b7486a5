"""Cases of the operators that stand between a decoder layer's quantized products.

Five operators: the root-mean-square norm with the residual's addition (`w4_rmsnorm*`), the gated
activation (`w4_silu_mul*`), rotary positions with the write into a paged cache (`w4_rope_cache`),
block tables and slot maps from request lengths (`w4_block_tables`) and attention of new tokens over
the paged cache (`w4_paged_attention`).  With `own` false a pass runs their plain form in elementary
torch operations, with `own` true the framework's calls.
"""

import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
EPS = 1e-5

# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------


def listed():
    return [
        # one decoded token's row between two 4-bit products: y of w4_gemv in, x of the next one out
        dict(name="norm one row", op="norm", rows=1, k=8192, x="f32", r="bf16", out="bf16"),
        # a prefill batch in front of an FP8 product
        dict(name="norm prefill fp8", op="norm", rows=4096, k=8192, x="bf16", r="bf16", out="fp8"),
        # the gate of a batch of decoded tokens, f32 from w4_gemv, bf16 for the next w4_gemv
        dict(name="gate decode", op="gate", rows=16, f=28672, x="f32", out="bf16"),
        # the gate of an odd prefill batch in front of an INT8 product
        dict(name="gate prefill int8", op="gate", rows=2049, f=11008, x="bf16", out="int8"),
        # a batch of decoded tokens far into long contexts, written into an E4M3 cache
        dict(name="rope decode fp8", op="rope", tokens=16, far=100000, heads=64, kv=8, d=128, rot=128, inter=False,
             scaling="bands", page=16, cache="fp8", x="f32"),
        # a prefill batch, interleaved pairs on half of each head, written into a bf16 cache
        dict(name="rope prefill", op="rope", tokens=4096, far=4096, heads=32, kv=32, d=128, rot=64, inter=True,
             scaling="none", page=64, cache="bf16", x="bf16"),
        # one decode step of a serving batch: one token more for every request
        dict(name="tables decode", op="tables", seqs=64, new=1, cached=8192, page=16),
        # a step that mixes prompts and decoded tokens
        dict(name="tables mixed", op="tables", seqs=256, new=64, cached=4096, page=64),
        # one request's next token over a short context: latency
        dict(name="attend one token", op="attend", seqs=1, new=1, cached=1000, heads=32, kv=32, d=128, page=16,
             cache="bf16", window=0),
        # a serving batch's decode step with ragged contexts
        dict(name="attend decode", op="attend", seqs=32, new=1, cached=8192, heads=64, kv=8, d=128, page=16,
             cache="bf16", window=0),
        # two requests at long contexts over an E4M3 cache
        dict(name="attend long fp8", op="attend", seqs=2, new=1, cached=100000, heads=64, kv=8, d=128, page=64,
             cache="fp8", window=0),
        # a chunk of a prompt over what is cached of it
        dict(name="attend chunk", op="attend", seqs=2, new=2048, cached=6144, heads=64, kv=8, d=128, page=32,
             cache="bf16", window=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "gate", "rope", "tables", "attend", "attend"))
    if op == "norm":
        k = 128 * _log(rng, 1, 128)
        return dict(op=op, rows=_log(rng, 1, min(4096, 4096 * 8192 // k)), k=k, x=rng.choice(("bf16", "f32")),
                    r=rng.choice(("bf16", "f32", "none")), out=rng.choice(("bf16", "f32", "fp8", "int8")))
    if op == "gate":
        f = 128 * _log(rng, 1, 224)
        return dict(op=op, rows=_log(rng, 1, min(4096, 2049 * 11008 // f)), f=f, x=rng.choice(("bf16", "f32")),
                    out=rng.choice(("bf16", "f32", "fp8", "int8")))
    d = rng.choice((64, 128))
    kv, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 8))
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 4096), far=_log(rng, 64, 1000000), heads=kv * group, kv=kv, d=d,
                    rot=16 * rng.randint(1, d // 16), inter=rng.random() < 0.5,
                    scaling=rng.choice(("none", "linear", "bands", "ramp")), page=2 ** rng.randint(4, 8),
                    cache=rng.choice(("bf16", "fp8")), x=rng.choice(("bf16", "f32")))
    if op == "tables":
        seqs = _log(rng, 1, 1024)
        return dict(op=op, seqs=seqs, new=_log(rng, 1, max(1, 16384 // seqs)), cached=_log(rng, 16, 8192),
                    page=2 ** rng.randint(4, 8))
    new = rng.choice((1, 1, _log(rng, 2, 16), _log(rng, 17, 1024)))
    cached = _log(rng, 1, 16384)
    most = max(1, int(2 * 2048 * 8192 * 64 // (new * (new + cached) * kv * group)))  # plain scores no larger than the largest's
    room = max(1, int(2 ** 28 // ((new + cached) * kv * d)))
    return dict(op=op, seqs=_log(rng, 1, max(1, min(64, most, room))), new=new, cached=cached, heads=kv * group, kv=kv, d=d,
                page=2 ** rng.randint(4, 8), cache=rng.choice(("bf16", "fp8")),
                window=rng.choice((0, 0, _log(rng, 1, 4096))))


def _lengths(case):
    """New and cached tokens of each request: the first has the most of both, the others are spread below."""
    n = case["seqs"]
    r = random.Random("%d %d %d" % (n, case["new"], case["cached"]))
    new = [case["new"]] + [r.randint(1, case["new"]) for _ in range(n - 1)]
    cached = [case["cached"]] + [r.randint(case["cached"] // 2, case["cached"]) for _ in range(n - 1)]
    return new, cached


def _visible(case):
    """Pairs of a query and a key that it sees, and keys that any query of their request sees."""
    new, cached = _lengths(case)
    w = case["window"]
    pairs = keys = 0
    for n, c in zip(new, cached):
        keys += n + c if not w else min(n + c, n + w - 1)
        if not w or w >= n + c:
            pairs += n * c + n * (n + 1) // 2
        else:
            first = max(0, min(n, w - c))  # queries whose window passes the start
            pairs += first * c + first * (first + 1) // 2 + (n - first) * w
    return pairs, keys


SIZE = {"f32": 4, "bf16": 2, "fp8": 1, "int8": 1, "none": 0}


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["k"]
        row = 4 * case["rows"] if SIZE[case["out"]] == 1 else 0
        return {"bytes": n * (SIZE[case["x"]] + 2 * SIZE[case["r"]] + SIZE[case["out"]]) + 2 * case["k"] + row,
                "flops": 6 * n}
    if op == "gate":
        n = case["rows"] * case["f"]
        row = 4 * case["rows"] if SIZE[case["out"]] == 1 else 0
        return {"bytes": n * (2 * SIZE[case["x"]] + SIZE[case["out"]]) + row, "flops": 6 * n}
    if op == "rope":
        t, d = case["tokens"], case["d"]
        cache = 2 * case["kv"] * (d * SIZE[case["cache"]] + (4 if case["cache"] == "fp8" else 0))
        return {"bytes": t * ((case["heads"] + 2 * case["kv"]) * d * SIZE[case["x"]] + case["heads"] * d * 2 + cache + 12)
                + 4 * case["rot"], "flops": t * (case["heads"] + case["kv"]) * case["rot"] * 3}
    if op == "tables":
        new, cached = _lengths(case)
        p, t = case["page"], sum(new)
        taken = sum((n + c + p - 1) // p - (c + p - 1) // p for n, c in zip(new, cached))
        return {"bytes": 16 * case["seqs"] + 8 * taken + 12 * t + 12, "flops": 0}
    pairs, keys = _visible(case)
    new, _ = _lengths(case)
    key = 2 * (case["d"] * SIZE[case["cache"]] + (4 if case["cache"] == "fp8" else 0))
    return {"bytes": keys * case["kv"] * key + 2 * sum(new) * case["heads"] * case["d"] * 2,
            "flops": 4 * pairs * case["heads"] * case["d"]}


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


def _rows_out(case, rows, k):
    """Buffers that a user's program keeps for the rows an operator writes."""
    if case["out"] in TYPE:
        return dict(y=torch.empty(rows, k, dtype=TYPE[case["out"]], device=DEV))
    return dict(codes=torch.empty(rows, k, dtype=torch.uint8 if case["out"] == "fp8" else torch.int8, device=DEV),
                scales=torch.empty(rows, dtype=torch.float32, device=DEV))


def _cache(case, pages, g=None):
    """A paged cache [pages, kv heads, page, d]: zeros, or filled with normal rows."""
    shape = (pages, case["kv"], case["page"], case["d"])
    fp8 = case["cache"] == "fp8"
    got = {}
    for n in ("k", "v"):
        if g is None:
            got[n] = torch.zeros(shape, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
            got[n + "_scales"] = torch.ones(shape[:3], device=DEV) if fp8 else None
            continue
        x = torch.randn(shape, device=DEV, generator=g, dtype=torch.bfloat16)
        got[n], got[n + "_scales"] = x, None
        if fp8:
            s = x.abs().amax(-1, keepdim=True).float() / E4M3_MAX
            got[n] = (x.float() / s).to(torch.float8_e4m3fn).view(torch.uint8)
            got[n + "_scales"] = s.squeeze(-1)
    return got


def _rope_spec(case):
    """Scalings as long-context models state them: trained on 8192 positions, stretched eight times."""
    s = dict(rotary_dim=case["rot"], base=500000.0, interleaved=case["inter"], scaling=case["scaling"])
    if case["scaling"] != "none":
        s["factor"] = 8.0
    if case["scaling"] == "bands":
        s.update(low=1.0, high=4.0, original_positions=8192)
    if case["scaling"] == "ramp":
        s.update(low=1.0, high=32.0, original_positions=8192)
    return s


def _frequencies(s):
    """Angle per position of each pair, and the amplitude of the rotation, on the host in 64 bits."""
    half = s["rotary_dim"] // 2
    f = [s["base"] ** (-i / half) for i in range(half)]
    kind = s["scaling"]
    if kind == "none":
        return f, 1.0
    if kind == "linear":
        return [x / s["factor"] for x in f], 1.0
    if kind == "bands":  # turns over the trained positions: few: stretched, many: kept, between: blended
        turns = [s["original_positions"] * x / (2 * math.pi) for x in f]
        keep = [min(1.0, max(0.0, (t - s["low"]) / (s["high"] - s["low"]))) for t in turns]
        return [x * (k + (1 - k) / s["factor"]) for x, k in zip(f, keep)], 1.0
    at = [half * math.log(s["original_positions"] / (2 * math.pi * t)) / math.log(s["base"]) for t in (s["high"], s["low"])]
    first, last = max(0, math.floor(at[0])), min(2 * half - 1, math.ceil(at[1]))
    if first == last:
        last += 0.001
    stretch = [min(1.0, max(0.0, (i - first) / (last - first))) for i in range(half)]
    return [x * (1 - r + r / s["factor"]) for x, r in zip(f, stretch)], 0.1 * math.log(s["factor"]) + 1.0


def _paged(case, g):
    """Block tables over shuffled pages for the requests' cached and new tokens."""
    new, cached = _lengths(case)
    p = case["page"]
    total = [n + c for n, c in zip(new, cached)]
    need = [(t + p - 1) // p for t in total]
    pages = sum(need) + 3
    order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
    wide = max(need)
    at = torch.arange(wide, device=DEV)
    start = torch.tensor([sum(need[:b]) for b in range(len(need))], device=DEV)
    used = at < torch.tensor(need, device=DEV)[:, None]
    table = torch.where(used, order[(start[:, None] + at).clamp_max(pages - 1)], -1).to(torch.int32)
    cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device=DEV)
    return dict(table=table.contiguous(), cu=cu, lens=torch.tensor(total, dtype=torch.int32, device=DEV), pages=pages,
                tokens=sum(new), most=max(new), longest=max(total))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    if op == "norm":
        rows, k = case["rows"], case["k"]
        s = dict(case=case, x=_rows(g, rows, k, TYPE[case["x"]]), weight=(1 + 0.1 * torch.randn(k, device=DEV, generator=g)).bfloat16(),
                 r=None, r_out=None, **_rows_out(case, rows, k))
        if case["r"] != "none":
            s["r"] = _rows(g, rows, k, TYPE[case["r"]])
            s["r_out"] = torch.empty_like(s["r"])
        return s
    if op == "gate":
        rows, f = case["rows"], case["f"]
        return dict(case=case, x=_rows(g, rows, 2 * f, TYPE[case["x"]], 5.0), **_rows_out(case, rows, f))
    if op == "rope":
        t, p = case["tokens"], case["page"]
        pages = (t + p - 1) // p + 2
        spec = _rope_spec(case)
        freqs, amplitude = _frequencies(spec)
        cache = _cache(case, pages)
        s = dict(case=case, cache=cache, amplitude=amplitude, freqs=torch.tensor(freqs, dtype=torch.float64, device=DEV),
                 x=_rows(g, t, (case["heads"] + 2 * case["kv"]) * case["d"], TYPE[case["x"]]),
                 positions=torch.randint(0, case["far"], (t,), device=DEV, generator=g).to(torch.int32),
                 slots=torch.randperm(pages * p, device=DEV, generator=g)[:t].contiguous(),
                 q=torch.empty(t, case["heads"], case["d"], dtype=torch.bfloat16, device=DEV))
        if own:
            import dequant_gemv_w4_amd as w4
            s["rope"] = w4.W4Rope.make(**spec)
            s["kv"] = w4.W4KVCache(**cache)
        return s
    if op == "tables":
        s = _paged(case, g)
        new, cached = _lengths(case)
        count = 4 * s["pages"]
        s.update(case=case, new=torch.tensor(new, dtype=torch.int32, device=DEV),
                 cached=torch.tensor(cached, dtype=torch.int32, device=DEV),
                 free=torch.randperm(count, device=DEV, generator=g).to(torch.int32),
                 count=torch.full((1,), count, dtype=torch.int32, device=DEV))
        s["out"] = dict(lens_out=torch.empty_like(s["cached"]), free_count_out=torch.empty_like(s["count"]),
                        cu_q=torch.empty_like(s["cu"]), positions=torch.empty(s["tokens"], dtype=torch.int32, device=DEV),
                        slots=torch.empty(s["tokens"], dtype=torch.int64, device=DEV))
        return s
    s = _paged(case, g)
    cache = _cache(case, s["pages"], g)
    shape = (s["tokens"], case["heads"], case["d"])
    s.update(case=case, cache=cache, scale=case["d"] ** -0.5, q=torch.randn(shape, device=DEV, generator=g).bfloat16(),
             o=torch.empty(shape, dtype=torch.bfloat16, device=DEV))
    if own:
        import dequant_gemv_w4_amd as w4
        s["kv"] = w4.W4KVCache(**cache)
        s["workspace"] = torch.empty(max(1, w4.w4_paged_attention_workspace_bytes(
            s["q"].shape[0], case["heads"], s["kv"], case["seqs"], s["table"].shape[1])), dtype=torch.uint8, device=DEV)
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------


def run(state):
    return (_run_own if own else _run_plain)(state)


def _as_values(case, codes, scales):
    """8-bit rows as the values of their codes: E4M3 bytes as they are, whole numbers in bf16 (which holds them)."""
    return [codes.view(torch.float8_e4m3fn) if codes.dtype == torch.uint8 else codes.to(torch.bfloat16), scales]


def _run_own(s):
    import dequant_gemv_w4_amd as w4
    case = s["case"]
    op = case["op"]
    if op == "norm":
        kept = dict(residual=s["r"], residual_out=s["r_out"])
        if case["out"] in TYPE:
            out = [w4.w4_rmsnorm(s["x"], s["weight"], EPS, y=s["y"], **kept)]
        else:
            call = w4.w4_rmsnorm_fp8 if case["out"] == "fp8" else w4.w4_rmsnorm_int8
            out = _as_values(case, *call(s["x"], s["weight"], EPS, codes=s["codes"], scales=s["scales"], **kept))
        return out + ([s["r_out"]] if s["r"] is not None else [])
    if op == "gate":
        if case["out"] in TYPE:
            return [w4.w4_silu_mul(s["x"], y=s["y"])]
        call = w4.w4_silu_mul_fp8 if case["out"] == "fp8" else w4.w4_silu_mul_int8
        return _as_values(case, *call(s["x"], codes=s["codes"], scales=s["scales"]))
    if op == "rope":
        w4.w4_rope_cache(s["x"], s["kv"], s["positions"], s["slots"], s["rope"], s["freqs"], q=s["q"])
        return _cache_out(case, s["q"], s["cache"])
    if op == "tables":
        o = s["out"]
        w4.w4_block_tables(s["new"], s["cached"], s["free"], s["count"], s["table"], case["page"], **o)
        return [o["cu_q"], o["positions"], o["slots"], o["lens_out"], o["free_count_out"], s["table"]]
    return [w4.w4_paged_attention(s["q"], s["kv"], s["table"], s["cu"], s["lens"], s["scale"], window=case["window"],
                                  o=s["o"], workspace=s["workspace"])]


def _cache_out(case, q, c):
    if case["cache"] == "bf16":
        return [q, c["k"], c["v"]]
    return [q, c["k"].view(torch.float8_e4m3fn), c["v"].view(torch.float8_e4m3fn), c["k_scales"], c["v_scales"]]


def _codes(y, kind):
    """8-bit rows of y: codes in their own type, and the scale of each row."""
    top = E4M3_MAX if kind == "fp8" else 127.0
    most = y.abs().amax(-1, keepdim=True)
    scale = torch.where(most == 0, 1.0, most / top)
    q = y / scale
    q = q.to(torch.float8_e4m3fn).view(torch.uint8) if kind == "fp8" else q.round().clamp(-128, 127).to(torch.int8)
    return q, scale.squeeze(-1)


def _rows_plain(case, y):
    return [y.to(TYPE[case["out"]])] if case["out"] in TYPE else _as_values(case, *_codes(y, case["out"]))


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        h, kept = s["x"].float(), []
        if s["r"] is not None:
            kept = [(h + s["r"].float()).to(s["r"].dtype)]
            h = kept[0].float()
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
        return _rows_plain(case, y) + kept
    if op == "gate":
        gate, up = s["x"].float().chunk(2, -1)
        return _rows_plain(case, gate / (1 + torch.exp(-gate)) * up)
    if op == "rope":
        return _plain_rope(s)
    if op == "tables":
        return _plain_tables(s)
    return _plain_attend(s)


def _plain_rope(s):
    case = s["case"]
    t, d, h, kv, half = case["tokens"], case["d"], case["heads"], case["kv"], case["rot"] // 2
    x = s["x"].float().view(t, h + 2 * kv, d)
    a = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = ((s["amplitude"] * f(a)).float()[:, None] for f in (torch.cos, torch.sin))
    turned = x[:, : h + kv]
    if case["inter"]:
        x0, x1 = turned[..., 0: 2 * half: 2], turned[..., 1: 2 * half: 2]
    else:
        x0, x1 = turned[..., :half], turned[..., half: 2 * half]
    y = turned.clone()
    y0, y1 = x0 * cos - x1 * sin, x0 * sin + x1 * cos
    if case["inter"]:
        y[..., 0: 2 * half: 2], y[..., 1: 2 * half: 2] = y0, y1
    else:
        y[..., :half], y[..., half: 2 * half] = y0, y1
    page, at = s["slots"] // case["page"], s["slots"] % case["page"]
    for n, rows in (("k", y[:, h:]), ("v", x[:, h + kv:])):
        if case["cache"] == "fp8":
            codes, scales = _codes(rows, "fp8")
            s["cache"][n][page, :, at] = codes
            s["cache"][n + "_scales"][page, :, at] = scales
        else:
            s["cache"][n][page, :, at] = rows.bfloat16()
    return _cache_out(case, y[:, :h].bfloat16(), s["cache"])


def _plain_tables(s):
    p, t = s["case"]["page"], s["tokens"]
    new, cached = s["new"].long(), s["cached"].long()
    have, want = (cached + p - 1) // p, (cached + new + p - 1) // p
    ends, taken = new.cumsum(0), (want - have).cumsum(0)
    cu = torch.cat((ends.new_zeros(1), ends))
    token = torch.arange(t, device=DEV)
    b = torch.searchsorted(ends, token, right=True)
    pos = cached[b] + token - cu[b]
    at = pos // p
    fresh = at >= have[b]
    count = s["count"].long()
    place = count - 1 - ((taken - (want - have))[b] + at - have[b])
    page = torch.where(fresh, s["free"].long()[torch.where(fresh, place, 0)], s["table"].long()[b, at])
    s["table"][b, at] = page.int()
    return [cu.int(), pos.int(), page * p + pos % p, (cached + new).int(), (count - taken[-1]).int(), s["table"]]


def _gathered(c, n, pages, at, dtype):
    """Keys or values of the requests [seqs, kv heads, longest, d] by pages and places in them."""
    x = c[n]
    if c[n + "_scales"] is None:
        return x[pages, :, at].to(dtype).transpose(1, 2).contiguous()
    codes = x.view(torch.uint8)[pages, :, at].view(torch.float8_e4m3fn).to(dtype)
    return (codes * c[n + "_scales"][pages, :, at].to(dtype)[..., None]).transpose(1, 2).contiguous()


def _plain_attend(s):
    case = s["case"]
    n, p, h, kv, d = case["seqs"], case["page"], case["heads"], case["kv"], case["d"]
    most, longest = s["most"], s["longest"]
    j = torch.arange(longest, device=DEV)
    pages = s["table"].long()[:, j // p].clamp_min(0)
    k, v = (_gathered_rows(s["cache"], x, pages, j % p) for x in ("k", "v"))
    cu, lens = s["cu"].long(), s["lens"].long()
    i = torch.arange(most, device=DEV)
    real = i < (cu[1:] - cu[:-1])[:, None]
    rows = torch.where(real, cu[:-1, None] + i, 0)
    q = s["q"][rows].float().view(n, most, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(n, kv, -1, d)
    z = torch.matmul(q, k.transpose(-1, -2).contiguous()).view(n, h, most, longest).mul_(s["scale"])
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + i
    seen = j <= pos[..., None]
    if case["window"]:
        seen &= j > pos[..., None] - case["window"]
    z.masked_fill_(~seen[:, None], -math.inf)
    z = z.sub_(z.amax(-1, keepdim=True).clamp_min(-3e38)).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(n, kv, -1, longest), v).view(n, h, most, d) / total
    return [o.transpose(1, 2)[real].bfloat16()]


def _gathered_rows(c, n, pages, at):
    return _gathered(c, n, pages, at.expand_as(pages), torch.float32)


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tables":
        return None
    if op in ("norm", "gate"):
        x, kept = s["x"].to(torch.float64), []
        if op == "norm":
            if case["r"] != "none":
                x = x + s["r"]
                kept = [x]
                x = x.to(s["r"].dtype).double()  # the norm is of the residual as it is stored
            y = s["weight"].double() * x / ((x * x).sum(1, keepdim=True) / case["k"] + EPS).sqrt()
        else:
            f = case["f"]
            y = torch.sigmoid(x[:, :f]) * x[:, :f] * x[:, f:]
        if case["out"] in TYPE:
            return [y] + kept
        step = y.abs().max(1).values / (448 if case["out"] == "fp8" else 127)
        codes = y / step[:, None]  # whole numbers for INT8; E4M3 codes are held against the quotients themselves
        return [codes if case["out"] == "fp8" else codes.round(), step] + kept
    if op == "rope":
        t, d, h, kv, rot = case["tokens"], case["d"], case["heads"], case["kv"], case["rot"]
        x = s["x"].double().view(t, -1, d).clone()
        z = torch.polar(torch.full((), s["amplitude"], dtype=torch.float64, device=DEV), torch.outer(s["positions"].double(), s["freqs"]))
        part = x[:, : h + kv, :rot]
        part = part.unflatten(-1, (-1, 2)) if case["inter"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
        turned = torch.view_as_real(torch.view_as_complex(part.contiguous()) * z[:, None])
        x[:, : h + kv, :rot] = (turned if case["inter"] else turned.transpose(-1, -2)).flatten(-2)
        out = [x[:, :h]]
        scales = []
        for first in (h, h + kv):
            rows = x[:, first: first + kv]
            step = rows.abs().max(-1).values / 448
            whole = torch.zeros(s["cache"]["k"].shape[0] * case["page"], kv, d, dtype=torch.float64, device=DEV)
            whole[s["slots"]] = rows if case["cache"] == "bf16" else rows / step[..., None]
            each = torch.ones(whole.shape[:2], dtype=torch.float64, device=DEV)
            each[s["slots"]] = step
            out.append(whole.unflatten(0, (-1, case["page"])).transpose(1, 2).contiguous())
            scales.append(each.unflatten(0, (-1, case["page"])).transpose(1, 2).contiguous())
        return out + (scales if case["cache"] == "fp8" else [])
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    group = case["heads"] // case["kv"]
    for b in range(case["seqs"]):
        length, n = lens[b], cu[b + 1] - cu[b]
        j = torch.arange(length, device=DEV)
        pages = s["table"][b].long()[j // case["page"]]
        pos = torch.arange(length - n, length, device=DEV)[:, None]
        hidden = (j > pos) | ((j <= pos - case["window"]) if case["window"] else (j < 0))
        for head in range(case["heads"]):
            k, v = (_one_head(s["cache"], x, pages, head // group, j % case["page"]) for x in ("k", "v"))
            z = (s["q"][cu[b]: cu[b + 1], head].double() @ k.t().contiguous()) * s["scale"]
            out[cu[b]: cu[b + 1], head] = torch.softmax(z.masked_fill_(hidden, -math.inf), -1) @ v
    return [out]


def _one_head(c, n, pages, head, at):
    x = c[n][pages, head, at]
    if c[n + "_scales"] is None:
        return x.double()
    return x.view(torch.float8_e4m3fn).double() * c[n + "_scales"][pages, head, at].double()[:, None]
