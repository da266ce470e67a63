"""Edges of the serving step and of 4-bit pages on the GPU: prompts written after a plan
that did not serve everyone, attention of packed rows by place, dims that do not turn, rows
dealt in two ways, and pages outside the pool."""
import numpy as np
import pytest
import torch

import long_context_chunked_gb300 as cp
import oracle
from paged4_helpers import check_decode4
from paged_helpers import Buffer, bf16_normal, i32
from test_gpu_paged import _ok
from test_gpu_step import FORMATS, Plan, _paged

pytestmark = pytest.mark.gpu


# ------------------------------------------- prompts written after a plan

WAITING = [  # held, new, free pages, table columns in use (page 16)
    ([33, 0, 0], [1, 100, 20], 3, 8),         # the second wants seven pages, and the third comes after it
    ([17, 30, 0], [3, 99, 15], 20, 8),        # the second has no room in its row of the table
    ([20, 5, -1], [12, 200, 9], 0, 16),       # nothing is free; the third place is empty
]


@FORMATS
@pytest.mark.parametrize("case", range(len(WAITING)))
def test_prompts_that_a_plan_did_not_serve_are_not_written(fmt, case):
    """Block tables that begin as zeros: the columns that a sequence would have got name
    page 0, which another one holds."""
    held, new, spare, cols = WAITING[case]
    rng = np.random.default_rng(case)
    nkv, hd, page = 2, 128, 16
    need = [-(-max(h, 0) // page) for h in held]
    c = _paged(fmt, nkv, hd, page, [page * (sum(need) + spare)], spare_pages=0)
    pages = c.pools[0].shape[0]
    c.table, c.cols = np.zeros((len(held), cols), np.int32), cols
    at = 0
    for b, n in enumerate(need):                          # (page 0 is the first sequence's first)
        c.table[b, :n] = np.arange(at, at + n)
        at += n
    c.fill(rng, np.maximum(held, 0))
    c.upload()
    free = list(range(at, pages))
    stack = Buffer(np.array(free + [-9] * (pages - len(free)), np.int32), torch.int32)
    rows = sum(n for h, n in zip(held, new) if h >= 0)
    x = [bf16_normal(rng, rows, nkv, hd) for _ in range(2)]
    d = [i32(v) for v in (held, new, [0] * 3, [0] * 4, [0] * rows, [0] * rows)]
    ctx = cp.Context(2 * nkv, nkv, hd, 1, 1, 1)
    ctx.paged_plan(c.kv, d[0], d[1], stack.t, i32([len(free)]), d[2], d[3], d[4], d[5])
    ctx.paged_write_kv(c.kv, d[0], *(Buffer(v, torch.bfloat16).t for v in x), row_starts=d[3], lens=d[2])
    assert ctx.sync_status() == cp.E_PAGE                 # (the plan's)
    lens, starts, _, _, fine = oracle.plan_ref(held, new, free, c.table, page, rows)
    assert not fine and d[2].tolist() == lens and d[3].tolist() == starts
    for b, (h, n) in enumerate(zip(held, lens)):
        if n > h >= 0:
            part = [v[starts[b]:starts[b + 1]] for v in x]
            oracle.paged_write_ref(c.pools, c.scales, c.table[b:], page, [h], [0, n - h], part)
    c.check_pools()
    assert c.intact()
    # a step of a token each, without row_starts
    step = [bf16_normal(rng, 3, nkv, hd) for _ in range(2)]
    have = [max(n - 1, -1) for n in lens]                 # (the last token of each again)
    upto = [n if b != 0 else n - 1 for b, n in enumerate(lens)]
    ctx.paged_write_kv(c.kv, i32(have), *(Buffer(v, torch.bfloat16).t for v in step), lens=i32(upto))
    _ok(ctx)
    have[0] = -1
    oracle.paged_write_ref(c.pools, c.scales, c.table, page, have, np.arange(4), step)
    c.check_pools()
    assert c.intact()


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
def test_packed_rows_are_attended_by_place(captured):
    """A step with an empty place, one without a new token, one with several and one that
    is not served: each served place's last new row."""
    rng = np.random.default_rng(5)
    nq, nkv, hd, page, held, new = 8, 2, 128, 16, [20, -1, 37, 0, 64, 11], [1, 9, 0, 3, 200, 30]
    need = [-(-max(h, 0) // page) for h in held]
    c = _paged("e2m1", nkv, hd, page, [page * (sum(need) + 5)], spare_pages=0)
    pages = c.pools[0].shape[0]
    c.table, c.cols = np.full((len(held), 8), 2 ** 30, np.int32), 8
    at = 0
    for b, n in enumerate(need):
        c.table[b, :n] = np.arange(at, at + n)
        at += n
    c.fill(rng, np.maximum(held, 0))
    c.upload()
    rows = sum(n for h, n in zip(held, new) if h >= 0)
    x = Buffer(bf16_normal(rng, rows, nq + 2 * nkv, hd), torch.bfloat16)
    ctx, nr = cp.Context(nq, nkv, hd, 1, 1, 1), cp.NormRope(1e4 ** (-np.arange(64) / 64))
    free = i32(list(range(at, pages)) + [0] * at)
    have, more, count, lens, starts, pos, slots = (
        i32(v) for v in (held, new, [pages - at], [0] * 6, [0] * 7, [0] * rows, [0] * rows))
    q = torch.zeros(rows, nq, hd, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros(6, nq, hd, dtype=torch.bfloat16, device="cuda"), torch.zeros(6, nq, device="cuda")
    ws = torch.empty(ctx.paged_decode_workspace(6), dtype=torch.uint8, device="cuda")

    def step():
        ctx.paged_plan(c.kv, have, more, free, count, lens, starts, pos, slots)
        ctx.norm_rope_write_kv(nr, c.kv, pos, slots, *x.t.split([nq, nkv, nkv], 1), q)
        ctx.paged_decode(c.kv, lens, q[starts[1:] - 1], out, ws, lse=lse)

    state = [t.clone() for t in (free, count, c.d_table.t)]
    step()
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t, was in zip((free, count, c.d_table.t), state):
            t.copy_(was)
        for t in (q, out, lse):
            t.zero_()
        graph.replay()
    assert ctx.sync_status() == cp.E_PAGE                 # (the fifth's columns end before its tokens)
    assert lens.tolist() == [21, -1, 37, 3, 64, 41]
    c.pools, c.scales, c.table = [d.host() for d in c.d_pools], [d.host() for d in c.d_scales], c.d_table.host()
    served = [0, 3, 5]
    c.table = c.table[served]
    last = [int(starts[b + 1]) - 1 for b in served]
    assert last == [0, 3, 233]
    check_decode4(c, q[last].double().cpu().numpy(), [21, 3, 41], hd ** -0.5, out[served].double().cpu().numpy(),
                  lse[served].double().cpu().numpy())


# ------------------------------------------- what does not turn

@pytest.mark.parametrize("appended", [False, True], ids=["dense", "bf16 pages"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("hd,rot", [(128, 24), (128, 0), (256, 64), (256, 0)])
def test_dims_that_do_not_turn_keep_to_themselves(hd, rot, interleaved, appended):
    """Without norm weights they are copies, bit for bit, whatever stands beside them: NaN,
    infinities and zeros of either sign.  With weights an infinity makes the root infinite,
    so every finite value 0."""
    rng = np.random.default_rng(hd + rot)
    rows, nq, nkv = 9, 4, 2
    x = bf16_normal(rng, rows, nq + nkv, hd)
    still = x[..., rot:]
    still[rng.random(still.shape) < 0.2] = 0x7F80
    still[rng.random(still.shape) < 0.2] = 0xFF80
    still[::2][rng.random(still[::2].shape) < 0.1] = 0x7FC1      # (of every second row)
    still[rng.random(still.shape) < 0.1] = 0x8000
    t = Buffer(x, torch.bfloat16)
    q, k = t.t[:, :nq], t.t[:, nq:]
    freq = 1e4 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    w = torch.ones(hd, device="cuda")
    pos, slots = i32(range(1, rows + 1)), i32(range(rows))
    ctx = cp.Context(nq, nkv, hd, 1, 1, 1)
    for normed in (False, True):
        nr = cp.NormRope(freq, *([w, w] if normed else []), interleaved=interleaved, device="cuda")
        q_out = torch.zeros(rows, nq, hd, dtype=torch.bfloat16, device="cuda")
        k_out = torch.zeros(rows, nkv, hd, dtype=torch.bfloat16, device="cuda")
        if appended:
            c = _paged("bf16", nkv, hd, 16, [rows]).upload()
            ctx.norm_rope_write_kv(nr, c.kv, pos, slots, q, k, k, q_out)
            k_out = c.d_pools[0].t[0, :, :rows].transpose(0, 1)
        else:
            ctx.norm_rope(nr, pos, q, k, q_out, k_out)
        _ok(ctx)
        got = np.concatenate([oracle.bf16_bits(y.contiguous().cpu()) for y in (q_out, k_out)], 1)
        if not normed:
            nan = (still & 0x7FFF) > 0x7F80
            assert np.array_equal(got[..., rot:][~nan], still[~nan])
            assert np.all((got[..., rot:][nan] & 0x7FFF) > 0x7F80)
            assert np.isfinite(oracle.bits_to_f64(got[..., :rot])).all()
        else:
            holds = lambda v: (((x & 0x7FFF) > 0x7F80) if v else ((x & 0x7FFF) == 0x7F80)).any(-1)  # noqa: E731
            infinite = holds(False) & ~holds(True)
            finite = infinite[..., None] & ((x & 0x7F80) != 0x7F80)
            assert finite.any() and np.all((got[finite] & 0x7FFF) == 0)


# ------------------------------------------- rows dealt to the GPU in two ways

@pytest.mark.parametrize("fmt", [None, "bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("nq,nkv,hd", [(1, 1, 256), (30, 2, 128), (32, 4, 128), (62, 2, 128), (28, 4, 256)], ids=str)
def test_rows_of_any_size_are_those_of_fewer_at_once(nq, nkv, hd, fmt):
    """Many rows, below and above the sizes from which blocks take rows in turn: the bits
    of calls of at most 2500."""
    rows = 7501
    gen = torch.Generator(device="cuda").manual_seed(nq)
    x = torch.randn(rows, nq + 2 * nkv, hd, generator=gen, device="cuda").to(torch.bfloat16).split([nq, nkv, nkv], 1)
    pos = torch.randint(-5, 10 ** 6, (rows,), generator=gen, device="cuda").int()
    slots = torch.randperm(rows, generator=gen, device="cuda").int()
    w = torch.rand(hd, generator=gen, device="cuda") + 0.5
    nr = cp.NormRope(1e4 ** (-np.arange(hd // 4) / (hd // 4)), w, w)
    ctx = cp.Context(nq, nkv, hd, 1, 1, 1)
    got = []
    for size in (rows, 2500):
        q = torch.zeros(rows, nq, hd, dtype=torch.bfloat16, device="cuda")
        k = torch.zeros(rows, nkv, hd, dtype=torch.bfloat16, device="cuda")
        c = None if fmt is None else _paged(fmt, nkv, hd, 64, [rows], seed=1).upload()
        for a in range(0, rows, size):
            part = slice(a, a + size)
            if c is None:
                ctx.norm_rope(nr, pos[part], x[0][part], x[1][part], q[part], k[part])
            else:
                ctx.norm_rope_write_kv(nr, c.kv, pos[part], slots[part], *(y[part] for y in x), q[part])
        _ok(ctx)
        got.append([q, k] if c is None else [q] + [b.t for b in c.d_pools + (c.d_scales or [])])
    for a, b in zip(*got):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)) and a.view(torch.uint8).any()


# ------------------------------------------- pages outside the pool

def test_trim_reports_pages_outside_the_pool():
    """They go to the list as they are, as the other pages do, and a plan that takes them
    from there reports them again and gives their rows no slot."""
    p = Plan([40, 20], 16, 3, 1, stride_pad=0)
    pages = len(p.free) + 5
    for bad in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        p = Plan([40, 20], 16, 3, 1, stride_pad=0)
        p.d_table.t[0, 1] = bad
        p.table[0, 1] = bad
        assert p.trim([40, 20], [40, 16]) == cp.OK                # (not among those that go back)
        assert p.trim([40, 16], [0, -1]) == cp.E_PAGE
        d = [i32(v) for v in ([0, 0], [32, 0], [0, 0], [0, 0, 0], [0] * 32, [0] * 32)]
        first, second = p.free[-1], p.free[-2]
        assert second == bad
        p.ctx.paged_plan(p.kv, d[0], d[1], p.d_free.t, p.d_count.t, d[2], d[3], d[4], d[5])
        assert p.ctx.sync_status() == cp.E_PAGE
        assert d[5].tolist() == [first * 16 + i for i in range(16)] + [-1] * 16
        assert p.d_free.intact() and p.d_table.intact() and p.d_count.intact()
    _ok(p.ctx)
