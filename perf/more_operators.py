"""What a serving step does around the attention, and the cache in 4 bits, as they are measured.

Five operators: ``plan`` (block tables, row starts, positions and slots of a step made from the
requests' lengths on the GPU, and the pages of tokens that are not kept given back),
``norm_rope`` (norms of queries and keys for each head with the position rotation in the same
pass), ``append`` (the same with the new tokens' K and V going straight into their pages),
``keep4`` (new tokens written to 4-bit pages and read back into the striped cache that the
chunked prefill extends) and ``decode4`` (attention of one new token per sequence over 4-bit
pages).

``run`` computes them in plain torch, or with ``own`` set through the framework's entry points.
"""
import math

import torch

own = False

BF16, E4M3 = "bf16", "e4m3"
E4M3_MAX = 448.0
TINY = 2.0 ** -110        # e4m3 pages: rows whose largest magnitude is below this are scaled as if it were this
GROUP = 32                # values of a 4-bit row that share a scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6
RAGGED_CACHE = "0,777,3000,8192,15000,60001"
RAGGED_ROWS = "4096,4096,1000,4096,37,4096"


def listed():
    dims = lambda nq, nkv, hd: dict(nq=nq, nkv=nkv, hd=hd)  # noqa: E731
    rope = lambda theta, rot, pairs="halves", norm="bf16": dict(theta=theta, rot=rot, pairs=pairs, norm=norm)  # noqa: E731
    return [
        # A decode step of a batch of chats, two of its places empty: a token each, a page for a few of them.
        dict(name="plan step 64", op="plan", page=16, spare=40, cols=512, rows=80, new=",".join(["1"] * 64),
             have=",".join(str(-1 if i in (9, 40) else (i * i * 37 + 911 * i) % 8192) for i in range(64))),
        # Whole prompts enter the cache.
        dict(name="plan prompts", op="plan", page=64, spare=100, cols=600, rows=64961, have="0,0,0,0,0",
             new="28672,4096,8192,15000,9001"),
        # The step of a handful of requests, one row each out of the projection's buffer.
        dict(name="norm rope step 7", op="norm_rope", at="499,0,15,4094,30,776,126976", fused=True, **rope(1e6, 256),
             **dims(32, 2, 256)),
        # The rows of a ragged batch of prompt chunks.
        dict(name="norm rope varlen", op="norm_rope", at=RAGGED_CACHE, rows=RAGGED_ROWS, fused=True, **rope(5e5, 128),
             **dims(32, 4, 128)),
        # The same step with its tokens appended to an 8-bit cache.
        dict(name="append step 7", op="append", format=E4M3, page=16, cached="500,1,16,4095,31,777,64", rows="1,1,1,1,1,1,1",
             fused=True, **rope(1e6, 256), **dims(32, 2, 256)),
        # The ragged chunks appended; half of each head rotated, neighbours paired.
        dict(name="append varlen e4m3", op="append", format=E4M3, page=64, cached=RAGGED_CACHE, rows=RAGGED_ROWS, fused=True,
             **rope(1e4, 64, "neighbours", "f32"), **dims(32, 4, 128)),
        # A long document and shorter ones, cache in bf16.
        dict(name="append 16k bf16", op="append", format=BF16, page=128, cached="0,0,0", rows="16384,777,3000", fused=False,
             **rope(1e6, 256), **dims(32, 2, 256)),
        # A second turn's prefix kept in 4 bits and handed to the chunked prefill.
        dict(name="keep4 32k", op="keep4", page=16, cached="0", rows="28672", shards=8, capacity=4096, v_f16=True,
             **dims(32, 2, 256)),
        # The ragged chunks.
        dict(name="keep4 varlen", op="keep4", page=64, cached="0,777,300,1,150,601", rows=RAGGED_ROWS, shards=8, capacity=613,
             v_f16=False, **dims(32, 4, 128)),
        # One short chat: latency is all that counts.
        dict(name="decode4 1x500", op="decode4", page=16, lens="500", **dims(8, 2, 128)),
        # One request with a long document.
        dict(name="decode4 1x128k", op="decode4", page=64, lens="126977", **dims(32, 2, 256)),
        # A serving batch: many requests of different ages.
        dict(name="decode4 64 ragged", op="decode4", page=16,
             lens=",".join(str(1 + (i * i * 37 + 911 * i) % 8192) for i in range(64)), **dims(32, 4, 128)),
    ]


def _between(rng, lo, hi):
    """Spread over the logarithm of the range; odd values as likely as even ones."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _text(values):
    return ",".join(map(str, values))


def draw(rng):
    op = rng.choice(["plan", "norm_rope", "append", "append", "keep4", "decode4", "decode4"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "plan":
        n = _between(rng, 1, 1024)
        new = [rng.choice([0, 1, 1, _between(rng, 1, max(1, 60000 // n))]) for _ in range(n)]
        have = [rng.choice([0, _between(rng, 1, 16384), _between(rng, 1, 2048)]) if rng.random() < 0.95 else -1 for _ in new]
        cols = -(-max(h + a for h, a in zip(have, new)) // page) + rng.choice([0, 3, 500])
        return dict(op=op, page=page, spare=rng.choice([0, 5, 1000]), cols=max(cols, 1), have=_text(have), new=_text(new),
                    rows=sum(a for h, a in zip(have, new) if h >= 0) + rng.choice([0, 1, 100]))
    hd = rng.choice([128, 256])
    nkv = rng.choice([1, 2, 4, 8] if hd == 128 else [1, 2, 4])
    group = rng.choice([1, 2, 3, 4, 6, 8, 16])
    c = dict(op=op, nq=nkv * group, nkv=nkv, hd=hd)
    if op == "decode4":
        top = _between(rng, 16, 65536)
        lens = [_between(rng, 1, top) if rng.random() < 0.97 else 0 for _ in range(_between(rng, 1, 96))]
        while len(lens) > 1 and len(lens) * max(lens) * nkv * hd > 130_000_000:
            lens.pop()
        return dict(c, page=page, lens=_text(lens))
    if rng.random() < 0.4:                           # a decode step
        rows = [1] * _between(rng, 1, 256)
    else:                                            # prompt chunks
        rows = [_between(rng, 1, 4096) for _ in range(_between(rng, 1, 16))]
        most = 30_000_000 // (nkv * hd) if op == "keep4" else 150_000_000 // ((c["nq"] + 2 * nkv) * hd)
        while len(rows) > 1 and sum(rows) > most:
            rows.pop()
    cached = [rng.choice([0, _between(rng, 1, 2048)]) for _ in rows]
    if op == "keep4":
        shards = rng.choice([1, 2, 3, 8])
        capacity = -(-max(a + b for a, b in zip(cached, rows)) // shards) + rng.choice([0, 5])
        if len(rows) * capacity * shards * nkv * hd > 500_000_000:
            rows, cached = rows[:16], cached[:16]
            capacity = -(-max(a + b for a, b in zip(cached, rows)) // shards)
        return dict(c, page=page, cached=_text(cached), rows=_text(rows), shards=shards, capacity=capacity, v_f16=rng.random() < 0.5)
    rot = rng.choice([hd, hd, hd // 2, 64, 24])
    c.update(theta=rng.choice([1e4, 5e5, 1e6]), rot=rot, pairs=rng.choice(["halves", "halves", "neighbours"]),
             norm=rng.choice(["bf16", "f32", "none"]), fused=rng.random() < 0.6)
    if op == "norm_rope":
        return dict(c, at=_text(rng.choice([x, x + _between(rng, 1, 1_000_000)]) for x in cached), rows=_text(rows))
    return dict(c, format=rng.choice([BF16, E4M3]), page=page, cached=_text(cached), rows=_text(rows))


def _ints(text):
    return [int(x) for x in text.split(",")]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _table(case, lens, gen):
    """A table that scatters the sequences over a pool with two pages to spare, and the pool's size."""
    need = [-(-n // case["page"]) for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(max(need), 1)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def _large_keys(x, gen):
    """One token in a hundred has a large key."""
    hit = torch.rand(x.shape[:-1], generator=gen, device="cuda") < 0.01
    return x * torch.where(hit, 2.0, 1.0).to(x.dtype).unsqueeze(-1)


def _inv_freq(case):
    return torch.tensor([case["theta"] ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)], dtype=torch.float64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "plan":
        return _prepare_plan(case, s, gen)
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    s["scale"] = 1.0 / math.sqrt(hd)
    if case["op"] == "decode4":
        lens = _ints(case["lens"])
        s["table"], pages = _table(case, lens, gen)
        shape = (pages, nkv, case["page"], hd)
        (s["kp"], s["ks"]), (s["vp"], s["vs"]) = _pack4(_large_keys(_normal(shape, gen), gen)), _pack4(_normal(shape, gen))
        s["lens"], s["q"] = _i32(lens), _normal((len(lens), nq, hd), gen)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((len(lens), nq), dtype=torch.float32, device="cuda")
    else:
        first = _ints(case["at"] if case["op"] == "norm_rope" else case["cached"])
        rows = _ints(case["rows"]) if "rows" in case else [1] * len(first)
        lens = [a + b for a, b in zip(first, rows)]
        total = sum(rows)
        starts = [0]
        for n in rows:
            starts.append(starts[-1] + n)
        s.update(cached=_i32(first), starts=_i32(starts), lens=_i32(lens), total=total)
        if case["op"] == "keep4":
            s["q"] = None
            s["k"], s["v"] = _large_keys(_normal((total, nkv, hd), gen), gen), _normal((total, nkv, hd), gen)
        else:
            qkv = _normal((total, nq + 2 * nkv, hd), gen)          # what the projection of the hidden states gives
            s["q"], s["k"], s["v"] = qkv.split([nq, nkv, nkv], 1)
            if not case["fused"]:
                s["q"], s["k"], s["v"] = (x.contiguous() for x in (s["q"], s["k"], s["v"]))
            seq = torch.repeat_interleave(torch.arange(len(rows), device="cuda"), _i32(rows), output_size=total)
            s["positions"] = s["cached"][seq] + torch.arange(total, device="cuda", dtype=torch.int32) - s["starts"][seq]
            s["q_out"] = torch.zeros((total, nq, hd), dtype=torch.bfloat16, device="cuda")
            wt = {"bf16": torch.bfloat16, "f32": torch.float32}.get(case["norm"])
            s["qw"], s["kw"] = (None if wt is None else (1 + 0.2 * _normal((hd,), gen, torch.float32)).to(wt) for _ in range(2))
            s["inv_freq"] = _inv_freq(case).cuda()
        if case["op"] == "norm_rope":
            s["k_out"] = torch.zeros((total, nkv, hd), dtype=torch.bfloat16, device="cuda")
        else:
            s["table"], pages = _table(case, lens, gen)
            shape = (pages, nkv, case["page"], hd)
            s["ks"] = s["vs"] = None
            if case["op"] == "keep4":
                (s["kp"], s["ks"]), (s["vp"], s["vs"]) = _pack4(_normal(shape, gen)), _pack4(_normal(shape, gen))
                cache = (len(rows), nkv, case["shards"], case["capacity"], hd)
                s["kc"] = torch.zeros(cache, dtype=torch.bfloat16, device="cuda")
                s["vc"] = torch.zeros(cache, dtype=torch.float16 if case["v_f16"] else torch.bfloat16, device="cuda")
            elif case["format"] == E4M3:
                (s["kp"], s["ks"]), (s["vp"], s["vs"]) = _quantise8(_normal(shape, gen)), _quantise8(_normal(shape, gen))
            else:
                s["kp"], s["vp"] = _normal(shape, gen), _normal(shape, gen)
            if case["op"] == "append":
                pos = s["positions"].long()
                s["slots"] = (s["table"][seq, pos // case["page"]] * case["page"] + pos % case["page"]).to(torch.int32)
    if own:
        import long_context_chunked_gb300 as cp
        s["ctx"] = cp.Context(nq, nkv, hd, case.get("shards", 1), case.get("capacity", 1), 1, s["scale"],
                              v_cache_f16=case.get("v_f16", False))
        if case["op"] in ("keep4", "decode4"):       # (bytes, as the pages hold them)
            s["kp"], s["vp"] = s["kp"].to(torch.uint8), s["vp"].to(torch.uint8)
        if "kp" in s:
            s["pages"] = cp.PagedKV(s["kp"], s["vp"], s["table"], s["ks"], s["vs"])
        if "inv_freq" in s:
            s["nr"] = cp.NormRope(_inv_freq(case), s["qw"], s["kw"], eps=EPS, interleaved=case["pairs"] == "neighbours")
        if case["op"] == "decode4":
            s["ws"] = torch.empty(s["ctx"].paged_decode_workspace(len(lens)), dtype=torch.uint8, device="cuda")
    return s


def _prepare_plan(case, s, gen):
    page, have, new = case["page"], _ints(case["have"]), _ints(case["new"])
    held = [-(-max(h, 0) // page) for h in have]
    want = [-(-(h + a) // page) - -(-h // page) if h >= 0 else 0 for h, a in zip(have, new)]
    pages, free = sum(held) + sum(want) + case["spare"], sum(want) + case["spare"]
    order = torch.randperm(max(pages, 1), generator=gen, device="cuda").to(torch.int32)
    b, cols = len(have), case["cols"]
    flat = torch.zeros(b * cols + 1, dtype=torch.int32, device="cuda")   # (the last one: nobody's)
    s["flat"], s["table"] = flat, flat[:-1].view(b, cols)
    at = free
    for i, n in enumerate(held):
        s["table"][i, :n] = order[at:at + n]
        at += n
    s["have"], s["new"] = _i32(have), _i32(new)
    s["free"] = torch.zeros(max(pages, 1) + 1, dtype=torch.int32, device="cuda")
    s["free"][:free] = order[:free]
    s["count"] = _i32([free])
    s["lens"], s["starts"] = torch.zeros_like(s["have"]), torch.zeros(b + 1, dtype=torch.int32, device="cuda")
    s["positions"], s["slots"] = (torch.zeros(case["rows"], dtype=torch.int32, device="cuda") for _ in range(2))
    if own:
        import long_context_chunked_gb300 as cp
        pool = torch.zeros((max(pages, 1), 1, page, 128), dtype=torch.bfloat16, device="cuda")
        s["ctx"] = cp.Context(1, 1, 128, 1, 1, 1)
        s["pages"] = cp.PagedKV(pool, pool, s["table"])
    return s


def _planned(s):
    return {"lens": s["lens"], "starts": s["starts"], "positions": s["positions"], "slots": s["slots"], "table": s["table"],
            "free": s["free"][:-1], "count": s["count"]}


def _pages(s):
    """The cache after new tokens were appended: e4m3 pages stand for their values, next to their scales."""
    out = {"q": s["q_out"], "k": s["kp"], "v": s["vp"]}
    if s["ks"] is not None:
        out.update(k_scales=s["ks"], v_scales=s["vs"])
    return out


def run(s):
    op = s["case"]["op"]
    if own:
        ctx = s["ctx"]
        if op == "plan":                       # a step, none of whose new tokens is kept
            ctx.paged_plan(s["pages"], s["have"], s["new"], s["free"][:-1], s["count"], s["lens"], s["starts"], s["positions"],
                           s["slots"])
            ctx.paged_trim(s["pages"], s["lens"], s["have"], s["free"][:-1], s["count"])
            return _planned(s)
        if op == "norm_rope":
            ctx.norm_rope(s["nr"], s["positions"], s["q"], s["k"], s["q_out"], s["k_out"])
            return {"q": s["q_out"], "k": s["k_out"]}
        if op == "append":
            ctx.norm_rope_write_kv(s["nr"], s["pages"], s["positions"], s["slots"], s["q"], s["k"], s["v"], s["q_out"])
            return _pages(s)
        if op == "keep4":
            ctx.paged_write_kv(s["pages"], s["cached"], s["k"], s["v"], row_starts=s["starts"])
            ctx.paged_read_kv(s["pages"], s["lens"], s["kc"], s["vc"], first=s["cached"])
            return {"k": s["kc"], "v": s["vc"]}
        ctx.paged_decode(s["pages"], s["lens"], s["q"], s["out"], s["ws"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    return {"plan": _plain_plan, "norm_rope": _plain_norm_rope, "append": _plain_append, "keep4": _plain_keep4,
            "decode4": _plain_decode4}[op](s)


# ---------------------------------------------------------------- the plain forms


def _quantise8(x):
    """e4m3 values and the fp32 scale of each row of the last axis: scale = amax / 448."""
    x = x.float()
    amax = x.abs().amax(-1).clamp_min(TINY)
    return (x * (E4M3_MAX / amax).unsqueeze(-1)).to(torch.float8_e4m3fn), amax / E4M3_MAX


def _scales4(x):
    """The two levels of a 4-bit row's scales (rows of the last axis, in x's type): s, a power of two with amax / s
    in [512, 1024), and r = e4m3(amax of the group / (6 s)) of each group."""
    amax = x.abs().amax(-1)
    s = torch.ldexp(torch.ones_like(amax), torch.frexp(amax.clamp_min(2.0 ** -117))[1] - 10)
    g = x.unflatten(-1, (-1, GROUP)).abs().amax(-1) / s[..., None]
    return s, (g / 6).to(torch.float8_e4m3fn).to(x.dtype)


def _codes4(y):
    """The nearest e2m1 code of |y|, ties to the even one: the borders lie between 0, .5, 1, 1.5, 2, 3, 4 and 6."""
    y = y.abs()
    return ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5))


def _pack4(x):
    """Rows as 4-bit pages hold them: two codes to a byte, the first in the lower half, and for each row its fp32 s and
    the e4m3 bytes of its groups."""
    x = x.float()
    s, r = _scales4(x)
    y = (x / s[..., None]).unflatten(-1, (-1, GROUP)) / r[..., None]
    y = torch.where(r[..., None] > 0, y, 0.0).flatten(-2)
    code = _codes4(y) + 8 * (y < 0)
    scales = torch.cat([s[..., None].contiguous().view(torch.uint8), r.to(torch.float8_e4m3fn).view(torch.uint8)], -1)
    return code[..., ::2] + 16 * code[..., 1::2], scales


def _values4(codes, scales):
    """fp32 rows of 4-bit pages."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    x = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    s, r = scales[..., :4].contiguous().view(torch.float32), scales[..., 4:].contiguous().view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (-1, GROUP)) * (s * r)[..., None]).flatten(-2)


def _plain_plan(s):
    page, table, free, count = s["case"]["page"], s["table"], s["free"], s["count"].long()
    n_seqs, cols = table.shape
    have, zero = s["have"].long(), torch.zeros(1, dtype=torch.int64, device="cuda")
    here = have >= 0
    new = torch.where(here, s["new"].long().clamp_min(0), 0)
    starts = torch.cat([zero, new.cumsum(0)])
    old = -(-have.clamp_min(0) // page)
    total = -(-(have.clamp_min(0) + new) // page)
    fits = here & (total <= cols)
    need = torch.where(fits, total - old, 0)
    upto = need.cumsum(0)
    granted = fits & ((need == 0) | (upto <= count))
    s["lens"].copy_(torch.where(granted, have + new, have))
    s["starts"].copy_(starts)
    # pages from the top of the free list, in order
    k = torch.arange(free.numel() - 1, device="cuda")
    taken = torch.where(granted, need, 0).sum()
    b = torch.searchsorted(upto, k, right=True).clamp_max(n_seqs - 1)
    to = torch.where(k < taken, b * cols + old[b] + k - (upto - need)[b], n_seqs * cols)
    s["flat"][to] = torch.where(k < taken, free[(count - 1 - k).clamp_min(0)], 0)
    # every row's place
    row = torch.arange(s["positions"].numel(), device="cuda")
    b = torch.searchsorted(starts[1:], row, right=True).clamp_max(n_seqs - 1)
    pos = have[b] + row - starts[b]
    some = (row < starts[-1]) & granted[b]
    at = table[b, torch.where(some, pos // page, 0)].long()
    s["positions"].copy_(torch.where(some, pos, -1))
    s["slots"].copy_(torch.where(some, at * page + pos % page, -1))
    # the new tokens are not kept: their pages go back
    left = count - taken
    keep, lens = have, s["lens"].long()
    kept = -(-keep.clamp_min(0) // page)
    gone = torch.where((keep >= 0) & (keep <= lens), -(-lens // page) - kept, 0)
    upto = gone.cumsum(0)
    back = gone.sum()
    b = torch.searchsorted(upto, k, right=True).clamp_max(n_seqs - 1)
    col = torch.where(k < back, kept[b] + k - (upto - gone)[b], 0)
    to = torch.where(k < back, left + back - 1 - k, free.numel() - 1)
    free[to] = torch.where(k < back, table[b, col], 0)
    s["count"].copy_(left + back)
    return _planned(s)


def _normed(x, weight, positions, inv_freq, case, wide=torch.float32):
    """Rows of heads [rows, heads, HD], normed and rotated, in the type `wide`."""
    x = x.to(wide)
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.to(wide)
    angle = positions.double()[:, None, None] * inv_freq                     # fp64: positions reach a million
    cos, sin = torch.cos(angle).to(wide), torch.sin(angle).to(wide)
    rot = case["rot"]
    if case["pairs"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_norm_rope(s):
    s["q_out"].copy_(_normed(s["q"], s["qw"], s["positions"], s["inv_freq"], s["case"]))
    s["k_out"].copy_(_normed(s["k"], s["kw"], s["positions"], s["inv_freq"], s["case"]))
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_append(s):
    case, page = s["case"], s["case"]["page"]
    s["q_out"].copy_(_normed(s["q"], s["qw"], s["positions"], s["inv_freq"], case))
    k = _normed(s["k"], s["kw"], s["positions"], s["inv_freq"], case)
    pid, slot = s["slots"].long() // page, s["slots"].long() % page
    for x, pool, scales in ((k, s["kp"], s["ks"]), (s["v"], s["vp"], s["vs"])):
        if case["format"] == E4M3:
            values, scale = _quantise8(x)
            pool.view(torch.uint8)[pid, :, slot] = values.view(torch.uint8)
            scales[pid, :, slot] = scale
        else:
            pool[pid, :, slot] = x.to(torch.bfloat16)
    return _pages(s)


def _plain_keep4(s):
    case, page = s["case"], s["case"]["page"]
    row = torch.arange(s["total"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["starts"], row, right=True) - 1
    pos = (s["cached"][seq] + row - s["starts"][seq]).long()
    pid, slot = s["table"][seq, pos // page].long(), pos % page
    for x, pool, scales, to in ((s["k"], s["kp"], s["ks"], s["kc"]), (s["v"], s["vp"], s["vs"], s["vc"])):
        pool[pid, :, slot], scales[pid, :, slot] = _pack4(x)
        to[seq, :, pos % case["shards"], pos // case["shards"]] = _values4(pool[pid, :, slot], scales[pid, :, slot]).to(to.dtype)
    return {"k": s["kc"], "v": s["vc"]}


def _plain_decode4(s):
    case = s["case"]
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    b, cols = s["table"].shape
    most = cols * case["page"]
    seen = (torch.arange(most, device="cuda") < s["lens"][:, None])[:, None, None]
    ids = s["table"].long()
    k, v = (_values4(p[ids], x[ids]).transpose(1, 2).reshape(b, nkv, most, hd) for p, x in ((s["kp"], s["ks"]), (s["vp"], s["vs"])))
    x = (s["q"].float().view(b, nkv, nq // nkv, hd) @ k.transpose(2, 3)) * s["scale"]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)       # a sequence without tokens
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).view(b, nq)
    return {"out": out.view(b, nq, hd).to(torch.bfloat16), "lse": lse}


# ---------------------------------------------------------------- what a pass has to do


def work(case):
    if case["op"] == "plan":
        have, new, page = _ints(case["have"]), _ints(case["new"]), case["page"]
        taken = sum(-(-(h + a) // page) - -(-h // page) for h, a in zip(have, new) if h >= 0)
        # lengths in, lengths and starts out; each row's position and slot; a page's number out of the list, into the
        # table, out of it and back
        return {"bytes": 4 * (4 * len(have) + 1) + 8 * case["rows"] + 16 * taken, "flops": 0}
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    row = nkv * hd                                   # values of K (or of V) per token
    held4 = 2 * nkv * (hd // 2 + 4 + hd // GROUP)    # a token's bytes in 4-bit pages
    if case["op"] == "decode4":
        lens = _ints(case["lens"])
        return {"bytes": sum(lens) * held4 + len(lens) * nq * (2 * hd * 2 + 4), "flops": 4 * hd * nq * sum(lens)}
    n = sum(_ints(case["rows"])) if "rows" in case else len(_ints(case["at"]))
    if case["op"] == "keep4":
        return {"bytes": n * (2 * row * 2 + 2 * held4 + 2 * row * 2), "flops": 0}
    # per value: square and sum, two factors, the rotation's two products
    flops = 8 * n * (nq + nkv) * hd
    if case["op"] == "norm_rope":
        return {"bytes": n * (4 + 2 * (nq + nkv) * hd * 2), "flops": flops}
    held = 2 * row * 2 if case["format"] == BF16 else 2 * (row + 4 * nkv)
    return {"bytes": n * (8 + 2 * nq * hd * 2 + 2 * row * 2 + held), "flops": flops}


# ---------------------------------------------------------------- the definitions in 64 bits


def _e4m3_of(x):
    """The nearest e4m3 value of each fp64 value (ties to even; at most 448)."""
    mag = x.abs().clamp_max(E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(mag.clamp_min(2.0 ** -6))).clamp(-6, 8) - 3)
    return torch.sign(x) * (torch.round(mag / step) * step).clamp_max(E4M3_MAX)


def _kept4(x):
    """The values that 4-bit pages hold for fp64 rows: each the nearest of s r times an e2m1 value."""
    amax = x.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -117)
    s = torch.exp2(torch.floor(torch.log2(amax)) - 9)
    s = torch.where(amax / s >= 1024, 2 * s, torch.where(amax / s < 512, s / 2, s))      # (where log2 was rounded)
    out = []
    for g in x.split(GROUP, -1):
        unit = s * _e4m3_of(g.abs().amax(-1, keepdim=True) / s / 6)
        y = (g / torch.where(unit > 0, unit, 1.0)).abs().clamp_max(6.0)
        step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
        out.append(torch.sign(g) * torch.round(y / step) * step * unit)
    return torch.cat(out, -1)


def _rotated(x, weight, positions, case):
    """Pair by pair: each is a complex number, turned by position * theta^(-2 i / rot)."""
    x, rot = x.double(), case["rot"]
    if weight is not None:
        x = x * weight.double() * torch.rsqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)
    first = torch.arange(rot // 2, device="cuda") * (1 if case["pairs"] == "halves" else 2)
    other = first + (rot // 2 if case["pairs"] == "halves" else 1)
    angle = positions.double()[:, None] * _inv_freq(case).cuda()
    z = torch.complex(x[..., first], x[..., other]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    out = x.clone()
    out[..., first], out[..., other] = z.real, z.imag
    return out


def _token4(codes, scales, table, page, g, n):
    """fp64 rows of kv head g, the first n tokens of one sequence."""
    t = torch.arange(n, device="cuda")
    pid, slot = table[t // page].long(), t % page
    byte, rec = codes[pid, g, slot].int(), scales[pid, g, slot]
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(1)
    e, m = (code >> 1) & 3, code & 1
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
    x = torch.where(code >= 8, -mag, mag)
    unit = rec[:, :4].contiguous().view(torch.float32).double() * rec[:, 4:].contiguous().view(torch.float8_e4m3fn).double()
    return x * unit.repeat_interleave(GROUP, 1)


def exact(case, seed):
    if case["op"] == "plan":             # whole numbers
        return None
    s = prepare(case, seed)
    nq, nkv, hd, page = case["nq"], case["nkv"], case["hd"], case.get("page")
    group = nq // nkv
    if case["op"] == "norm_rope":
        return {x: _rotated(s[x], s[x + "w"], s["positions"], case) for x in "qk"}
    if case["op"] == "append":
        got = {"q": _rotated(s["q"], s["qw"], s["positions"], case)}
        for name, x in (("k", _rotated(s["k"], s["kw"], s["positions"], case)), ("v", s["v"].double())):
            pool, scales = s[name + "p"].double(), s[name + "s"]
            at = s["slots"].long()
            if scales is not None:
                amax = x.abs().amax(-1).clamp_min(TINY)
                scales = scales.double()
                scales[at // page, :, at % page] = amax / E4M3_MAX
                x = _e4m3_of(x * (E4M3_MAX / amax)[..., None])
                got[name + "_scales"] = scales
            pool[at // page, :, at % page] = x
            got[name] = pool
        return got
    if case["op"] == "keep4":
        got = {}
        for name, to in (("k", s["kc"]), ("v", s["vc"])):
            x, out, at = _kept4(s[name].double()), torch.zeros(to.shape, dtype=torch.float64, device="cuda"), 0
            for b, (have, n) in enumerate(zip(_ints(case["cached"]), _ints(case["rows"]))):
                t = torch.arange(have, have + n, device="cuda")
                out[b, :, t % case["shards"], t // case["shards"]] = x[at:at + n].transpose(0, 1)
                at += n
            got[name] = out
        return got
    lens = _ints(case["lens"])
    out = torch.zeros((len(lens), nq, hd), dtype=torch.float64, device="cuda")
    lse = torch.full((len(lens), nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        for g in range(nkv if n else 0):
            h = slice(g * group, (g + 1) * group)
            x = s["q"][b, h].double() @ _token4(s["kp"], s["ks"], s["table"][b], page, g, n).T / math.sqrt(hd)
            lse[b, h] = torch.logsumexp(x, -1)
            out[b, h] = torch.exp(x - lse[b, h, None]) @ _token4(s["vp"], s["vs"], s["table"][b], page, g, n)
    return {"out": out, "lse": lse}
