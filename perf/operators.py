"""The paged KV cache and the packed prompt attention, as they are measured.

Four operators: ``paged_write`` (new tokens' K and V into a paged cache, in bf16 or
quantised to e4m3 with one scale per token and kv head), ``paged_read`` (pages back into the
striped cache that the chunked prefill reads), ``paged_decode`` (attention of one new token
per sequence over the pages) and ``prompt`` (causal attention of whole prompts, packed
one behind the other).

``run`` computes them in plain torch, or with ``own`` set through the framework's entry points.
"""
import math

import torch

own = False

BF16, E4M3 = "bf16", "e4m3"
E4M3_MAX = 448.0
TINY = 2.0 ** -110        # rows whose largest magnitude is below this are scaled as if it were this


def listed():
    dims = lambda nq, nkv, hd: dict(nq=nq, nkv=nkv, hd=hd)  # noqa: E731
    varlen_cache = "0,777,3000,8192,15000,60001"
    varlen_chunk = "4096,4096,1000,4096,37,4096"
    return [
        # A decode step of a handful of requests: each appends one token to its cache.
        dict(name="write step 7", op="paged_write", format=E4M3, page=16, cached="500,1,16,4095,31,777,64",
             rows="1,1,1,1,1,1,1", **dims(32, 2, 256)),
        # Prompt chunks of a ragged batch, quantised as they enter the cache.
        dict(name="write varlen e4m3", op="paged_write", format=E4M3, page=64, cached="0,777,3000,8192,1500,601",
             rows=varlen_chunk, **dims(32, 4, 128)),
        # Whole prompts of a long-context batch, kept in bf16.
        dict(name="write prompts bf16", op="paged_write", format=BF16, page=128, cached="0,0,0,0,0",
             rows="28672,4096,8192,15000,9001", **dims(32, 2, 256)),
        # A request comes back for a second turn: its prefix is read for the chunked prefill.
        dict(name="read 32k prefix e4m3", op="paged_read", format=E4M3, page=16, lens="28672", shards=8,
             capacity=4096, v_f16=True, **dims(32, 2, 256)),
        # The same for a ragged batch with a bf16 cache.
        dict(name="read varlen bf16", op="paged_read", format=BF16, page=64, lens=varlen_cache, shards=8,
             capacity=8013, v_f16=False, **dims(32, 4, 128)),
        # One short chat: latency is all that counts.
        dict(name="decode 1x500 bf16", op="paged_decode", format=BF16, page=16, lens="500", **dims(8, 2, 128)),
        # One request with a long document.
        dict(name="decode 1x128k e4m3", op="paged_decode", format=E4M3, page=64, lens="126977", **dims(32, 2, 256)),
        # A serving batch: many requests of different ages.
        dict(name="decode 64 ragged e4m3", op="paged_decode", format=E4M3, page=16,
             lens=",".join(str(1 + (i * i * 37 + 911 * i) % 8192) for i in range(64)), **dims(32, 4, 128)),
        # A batch of long contexts, cache in bf16.
        dict(name="decode 8x32k bf16", op="paged_decode", format=BF16, page=128,
             lens=",".join(["32768"] * 8), **dims(32, 2, 256)),
        # A few short questions prefilled together.
        dict(name="prompt short", op="prompt", lens="37,5,128,1,300", v_f16=True, **dims(8, 2, 128)),
        # The ragged batch of prompt lengths.
        dict(name="prompt varlen", op="prompt", lens=varlen_chunk, v_f16=True, **dims(32, 4, 128)),
        # One long document next to shorter ones.
        dict(name="prompt 16k", op="prompt", lens="16384,777,3000", v_f16=True, **dims(32, 2, 256)),
    ]


def _between(rng, lo, hi):
    """Spread over the logarithm of the range; odd values as likely as even ones."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["paged_write", "paged_read", "paged_decode", "paged_decode", "prompt"])
    hd = rng.choice([128, 256])
    nkv = rng.choice([1, 2, 4, 8] if hd == 128 else [1, 2, 4])
    group = rng.choice([1, 2, 3, 4, 6, 8, 16])
    c = dict(op=op, nq=nkv * group, nkv=nkv, hd=hd)
    per_token = nkv * hd
    if op == "prompt":
        n = _between(rng, 1, 24)
        most = 125_000_000_000 // (c["nq"] * hd)       # visible (query, key) pairs
        lens = [_between(rng, 1, 4096) for _ in range(n)]
        while len(lens) > 1 and sum(x * x for x in lens) > 2 * most:
            lens.pop()
        return dict(c, lens=",".join(map(str, lens)), v_f16=rng.random() < 0.7)
    c.update(format=rng.choice([BF16, E4M3]), page=rng.choice([16, 32, 64, 128, 256]))
    if op == "paged_write":
        if rng.random() < 0.4:                       # a decode step
            n = _between(rng, 1, 256)
            rows = [1] * n
        else:                                        # prompt chunks
            n = _between(rng, 1, 16)
            rows = [_between(rng, 1, 4096) for _ in range(n)]
            while len(rows) > 1 and sum(rows) * per_token > 30_000_000:
                rows.pop()
        cached = [rng.choice([0, _between(rng, 1, 2048)]) for _ in rows]
        return dict(c, rows=",".join(map(str, rows)), cached=",".join(map(str, cached)))
    if op == "paged_read":
        lens = [_between(rng, 1, 16384) for _ in range(_between(rng, 1, 16))]
        while len(lens) > 1 and sum(lens) * per_token > 30_000_000:
            lens.pop()
        shards = rng.choice([1, 2, 3, 8])
        capacity = -(-max(lens) // shards) + rng.choice([0, 5])
        return dict(c, lens=",".join(map(str, lens)), shards=shards, capacity=capacity, v_f16=rng.random() < 0.5)
    top = _between(rng, 16, 65536)
    lens = [_between(rng, 1, top) if rng.random() < 0.97 else 0 for _ in range(_between(rng, 1, 96))]
    while len(lens) > 1 and len(lens) * max(lens) * per_token > 130_000_000:
        lens.pop()
    return dict(c, lens=",".join(map(str, lens)))


def _ints(text):
    return [int(x) for x in text.split(",")]


def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _pool(case, lens, gen):
    """Page pools full of earlier requests' tokens, and a table that scatters the sequences over them."""
    page, nkv, hd = case["page"], case["nkv"], case["hd"]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(max(need), 1)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    pools, scales = [], []
    for is_k in (True, False):
        x = _normal((pages, nkv, page, hd), gen)
        if is_k:     # one token in a hundred has a large key
            x *= torch.where(torch.rand((pages, 1, page, 1), generator=gen, device="cuda") < 0.01, 2.0, 1.0).to(x.dtype)
        if case["format"] == E4M3:
            values, scale = _quantise(x)
            pools.append(values)
            scales.append(scale)
        else:
            pools.append(x)
            scales.append(None)
    return pools, scales, table


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    scale = 1.0 / math.sqrt(hd)
    s = {"case": case, "scale": scale}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] == "prompt":
        lens = _ints(case["lens"])
        rows = sum(lens)
        s.update(lens=lens, q=_normal((rows, nq, hd), gen), k=_normal((rows, nkv, hd), gen),
                 v=_normal((rows, nkv, hd), gen), out=torch.zeros((rows, nq, hd), dtype=torch.bfloat16, device="cuda"))
        if own:
            import long_context_chunked_gb300 as cp
            s["ctx"] = cp.Context(nq, nkv, hd, 1, 1, 1, scale, v_cache_f16=case["v_f16"])
            s["ws"] = torch.empty(s["ctx"].prefill_packed_workspace(lens), dtype=torch.uint8, device="cuda")
        return s
    if case["op"] == "paged_write":
        cached, rows = _ints(case["cached"]), _ints(case["rows"])
        lens = [a + b for a, b in zip(cached, rows)]
        starts = [0]
        for n in rows:
            starts.append(starts[-1] + n)
        k, v = (_normal((starts[-1], nkv, hd), gen) for _ in range(2))
        # A step appends one token to every sequence: its rows need no table of starts.
        s.update(cached=i32(cached), starts=None if max(rows) == 1 == min(rows) else i32(starts), k=k, v=v)
    else:
        lens = _ints(case["lens"])
        s.update(lens=i32(lens), total=sum(lens))
    (s["kp"], s["vp"]), (s["ks"], s["vs"]), s["table"] = _pool(case, lens, gen)
    shards, capacity = case.get("shards", 1), case.get("capacity", 1)
    if case["op"] == "paged_read":
        shape = (len(lens), nkv, shards, capacity, hd)
        s["kc"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        s["vc"] = torch.zeros(shape, dtype=torch.float16 if case["v_f16"] else torch.bfloat16, device="cuda")
    if case["op"] == "paged_decode":
        s["q"] = _normal((len(lens), nq, hd), gen)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((len(lens), nq), dtype=torch.float32, device="cuda")
    if own:
        import long_context_chunked_gb300 as cp
        s["ctx"] = cp.Context(nq, nkv, hd, shards, capacity, 1, scale, v_cache_f16=case.get("v_f16", False))
        s["pages"] = cp.PagedKV(s["kp"], s["vp"], s["table"], s["ks"], s["vs"])
        if case["op"] == "paged_decode":
            s["ws"] = torch.empty(s["ctx"].paged_decode_workspace(len(lens)), dtype=torch.uint8, device="cuda")
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        if op == "prompt":
            s["ctx"].prefill_packed(s["lens"], s["q"], s["k"], s["v"], s["out"], s["ws"])
            return s["out"]
        if op == "paged_write":
            s["ctx"].paged_write_kv(s["pages"], s["cached"], s["k"], s["v"], row_starts=s["starts"])
            return _pages(s)
        if op == "paged_read":
            s["ctx"].paged_read_kv(s["pages"], s["lens"], s["kc"], s["vc"])
            return {"k": s["kc"], "v": s["vc"]}
        s["ctx"].paged_decode(s["pages"], s["lens"], s["q"], s["out"], s["ws"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    return {"prompt": _plain_prompt, "paged_write": _plain_write, "paged_read": _plain_read, "paged_decode": _plain_decode}[op](s)


# ---------------------------------------------------------------- the plain forms


def _pages(s):
    """The cache after a write: e4m3 pages stand for their values, next to their scales."""
    out = {"k": s["kp"], "v": s["vp"]}
    if s["ks"] is not None:
        out.update(k_scales=s["ks"], v_scales=s["vs"])
    return out


def _quantise(x):
    """e4m3 values and the fp32 scale of each row of the last axis: scale = amax / 448."""
    x = x.float()
    amax = x.abs().amax(-1).clamp_min(TINY)
    return (x * (E4M3_MAX / amax).unsqueeze(-1)).to(torch.float8_e4m3fn), amax / E4M3_MAX


def _plain_write(s):
    case, page = s["case"], s["case"]["page"]
    row = torch.arange(s["k"].shape[0], device="cuda", dtype=torch.int32)
    if s["starts"] is None:
        seq, pos = row.long(), s["cached"].long()
    else:
        seq = torch.searchsorted(s["starts"], row, right=True) - 1
        pos = (s["cached"][seq] + row - s["starts"][seq]).long()
    pid, slot = s["table"][seq, pos // page].long(), pos % page
    for x, pool, scales in ((s["k"], s["kp"], s["ks"]), (s["v"], s["vp"], s["vs"])):
        if case["format"] == E4M3:
            values, scale = _quantise(x)
            pool.view(torch.uint8)[pid, :, slot] = values.view(torch.uint8)
            scales[pid, :, slot] = scale
        else:
            pool[pid, :, slot] = x
    return _pages(s)


def _values(pool, scales):
    """Rows of pages as fp32."""
    return pool.float() if scales is None else pool.float() * scales.unsqueeze(-1)


def _plain_read(s):
    case, page = s["case"], s["case"]["page"]
    lens = s["lens"].long()
    seq = torch.repeat_interleave(torch.arange(lens.numel(), device="cuda"), lens, output_size=s["total"])
    pos = torch.arange(s["total"], device="cuda") - (lens.cumsum(0) - lens)[seq]
    pid, slot = s["table"][seq, pos // page].long(), pos % page
    for pool, scales, to in ((s["kp"], s["ks"], s["kc"]), (s["vp"], s["vs"], s["vc"])):
        # (rows as 16- or 8-bit words are gathered, then widened)
        rows = pool.view(torch.uint8)[pid, :, slot].view(pool.dtype)
        rows = _values(rows, None if scales is None else scales[pid, :, slot])
        to[seq, :, pos % case["shards"], pos // case["shards"]] = rows.to(to.dtype)
    return {"k": s["kc"], "v": s["vc"]}


def _gathered(s, pool, scales, most):
    """[B, NKV, most, HD] fp32 of every sequence's first `most` tokens (padding: the table's other pages)."""
    b, nkv, hd = s["table"].shape[0], s["case"]["nkv"], s["case"]["hd"]
    ids = s["table"][:, :-(-most // s["case"]["page"])].long()
    x = _values(pool.view(torch.uint8)[ids].view(pool.dtype), None if scales is None else scales[ids])
    return x.transpose(1, 2).reshape(b, nkv, -1, hd)[:, :, :most]


def _plain_decode(s):
    case = s["case"]
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    most = s["table"].shape[1] * case["page"]
    b = s["q"].shape[0]
    q = s["q"].float().view(b, nkv, nq // nkv, hd)
    seen = (torch.arange(most, device="cuda") < s["lens"][:, None])[:, None, None]
    x = (q @ _gathered(s, s["kp"], s["ks"], most).transpose(2, 3)) * s["scale"]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)       # a sequence without tokens
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen.transpose(2, 3), _gathered(s, s["vp"], s["vs"], most), 0.0)
    out = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).view(b, nq)
    return {"out": out.view(b, nq, hd).to(torch.bfloat16), "lse": lse}


def _plain_prompt(s):
    case = s["case"]
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    out, at = torch.empty_like(s["out"]), 0
    for n in s["lens"]:
        q = s["q"][at:at + n].float().view(n, nkv, nq // nkv, hd).permute(1, 2, 0, 3)
        k, v = (s[x][at:at + n].float().transpose(0, 1) for x in "kv")
        for g in range(nkv):
            for r in range(0, n, 4096):                                  # blocks of rows, so that the scores fit
                m = min(n, r + 4096)
                x = (q[g, :, r:m] @ k[g, :m].T) * s["scale"]
                later = torch.arange(m, device="cuda") > torch.arange(r, m, device="cuda")[:, None]
                x = x.masked_fill_(later, -math.inf)
                p = torch.exp(x.sub_(x.amax(-1, keepdim=True)))
                o = (p @ v[g, :m]) / p.sum(-1, keepdim=True)
                out[at + r:at + m, g * (nq // nkv):(g + 1) * (nq // nkv)] = o.transpose(0, 1).to(torch.bfloat16)
        at += n
    return out


# ---------------------------------------------------------------- what a pass has to do


def work(case):
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    row = nkv * hd                                   # values of K (or of V) per token
    if case["op"] == "prompt":
        lens = _ints(case["lens"])
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": sum(lens) * (2 * nq * hd + 2 * row) * 2, "flops": 4 * hd * nq * pairs}
    held = 2 * row * 2 if case["format"] == BF16 else 2 * (row + 4 * nkv)   # a token's bytes in the cache
    if case["op"] == "paged_write":
        n = sum(_ints(case["rows"]))
        return {"bytes": n * (2 * row * 2 + held), "flops": 0}
    n = sum(_ints(case["lens"]))
    if case["op"] == "paged_read":
        return {"bytes": n * (held + 2 * row * 2), "flops": 0}
    b = len(_ints(case["lens"]))
    return {"bytes": n * held + b * nq * (2 * hd * 2 + 4), "flops": 4 * hd * nq * n}


# ---------------------------------------------------------------- the definitions in 64 bits


def _e4m3_of(x):
    """The nearest e4m3 value of each fp64 value (ties to even; at most 448)."""
    mag = x.abs().clamp_max(E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(mag.clamp_min(2.0 ** -6))).clamp(-6, 8) - 3)
    return torch.sign(x) * (torch.round(mag / step) * step).clamp_max(E4M3_MAX)


def _token(pool, scales, table, page, g, t0, t1):
    """fp64 rows of kv head g, tokens [t0, t1) of one sequence."""
    t = torch.arange(t0, t1, device="cuda")
    pid, slot = table[t // page].long(), t % page
    x = pool[:, g].reshape(-1, pool.shape[-1]).view(torch.uint8).view(pool.shape[0] * page, -1)[pid * page + slot]
    x = x.view(pool.dtype).double()
    return x if scales is None else x * scales[pid, g, slot].double()[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    group, scale = nq // nkv, 1.0 / math.sqrt(hd)
    page = case.get("page")
    if case["op"] == "paged_write":
        names = {"k": (s["k"], s["kp"], s["ks"]), "v": (s["v"], s["vp"], s["vs"])}
        got = {}
        for name, (x, pool, scales) in names.items():
            got[name] = pool.double()
            if scales is not None:
                got[name + "_scales"] = scales.double()
            at = 0
            for b, (have, n) in enumerate(zip(_ints(case["cached"]), _ints(case["rows"]))):
                t = torch.arange(have, have + n, device="cuda")
                pid, slot = s["table"][b, t // page].long(), t % page
                rows = x[at:at + n].double()
                if scales is not None:
                    amax = rows.abs().amax(-1).clamp_min(TINY)
                    got[name + "_scales"][pid, :, slot] = amax / E4M3_MAX
                    rows = _e4m3_of(rows * (E4M3_MAX / amax)[..., None])
                got[name][pid, :, slot] = rows
                at += n
        return got
    if case["op"] == "paged_read":
        k, v = torch.zeros(s["kc"].shape, dtype=torch.float64, device="cuda"), torch.zeros(s["vc"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_ints(case["lens"])):
            t = torch.arange(n, device="cuda")
            for g in range(nkv):
                k[b, g, t % case["shards"], t // case["shards"]] = _token(s["kp"], s["ks"], s["table"][b], page, g, 0, n)
                v[b, g, t % case["shards"], t // case["shards"]] = _token(s["vp"], s["vs"], s["table"][b], page, g, 0, n)
        return {"k": k, "v": v}
    if case["op"] == "paged_decode":
        lens = _ints(case["lens"])
        out = torch.zeros((len(lens), nq, hd), dtype=torch.float64, device="cuda")
        lse = torch.full((len(lens), nq), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            if n == 0:
                continue
            for g in range(nkv):
                h = slice(g * group, (g + 1) * group)
                x = s["q"][b, h].double() @ _token(s["kp"], s["ks"], s["table"][b], page, g, 0, n).T * scale
                lse[b, h] = torch.logsumexp(x, -1)
                out[b, h] = torch.exp(x - lse[b, h, None]) @ _token(s["vp"], s["vs"], s["table"][b], page, g, 0, n)
        return {"out": out, "lse": lse}
    if work(case)["flops"] > 8e12:       # fp64 products of more than that take too long
        return None
    out, at = torch.zeros((s["q"].shape[0], nq, hd), dtype=torch.float64, device="cuda"), 0
    for n in s["lens"]:
        for h in range(nq):
            k, v = s["k"][at:at + n, h // group].double(), s["v"][at:at + n, h // group].double()
            for r in range(0, n, 2048):
                m = min(n, r + 2048)
                x = s["q"][at + r:at + m, h].double() @ k[:m].T * scale
                x += torch.full((m - r, m), -math.inf, dtype=torch.float64, device="cuda").triu(r + 1)
                out[at + r:at + m, h] = torch.softmax(x, -1) @ v[:m]
        at += n
    return out
