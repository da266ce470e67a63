"""A serving step around the attention on the GPU against the oracle: plans and
trims of the paged cache (equal), norms and rotations of heads and appending to
the pages (within derived bounds), and the whole step captured and replayed."""
import numpy as np
import pytest
import torch

import long_context_chunked_gb300 as cp
import oracle
from paged4_helpers import Paged4, check_decode4
from paged_helpers import Buffer, Paged, bf16_normal, check_decode, i32
from test_gpu_paged import _ok

pytestmark = pytest.mark.gpu

FORMATS = pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e2m1"])


def _paged(fmt, nkv, hd, page, caps, **kw):
    return Paged4(nkv, hd, page, caps, **kw) if fmt == "e2m1" else Paged(nkv, hd, page, caps, fmt == "e4m3", **kw)


def _bits(x):
    return oracle.bf16_bits(torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16))


# --------------------------------------------------------------- plan and trim

class Plan:
    """Device state of a plan between canary bands, and the oracle's."""

    def __init__(self, have, page, cols, spare, seed=0, stride_pad=1):
        rng = np.random.default_rng(seed)
        held = [-(-max(h, 0) // page) for h in have]
        pages = max(sum(held) + spare, 1)
        order = [int(x) for x in rng.permutation(pages)]
        self.free, used = order[:pages - sum(held)], order[pages - sum(held):]
        self.table = np.full((len(have), cols + stride_pad), -7, np.int32)
        for b, n in enumerate(held):
            self.table[b, :n] = [used.pop() for _ in range(n)]
        self.page, self.cols, self.have = page, cols, np.asarray(have, np.int32)
        pool = torch.zeros(pages, 1, page, 128, dtype=torch.bfloat16, device="cuda")
        self.d_table = Buffer(self.table, torch.int32)
        stack = np.full(pages, -9, np.int32)
        stack[:len(self.free)] = self.free
        self.d_free, self.d_count = Buffer(stack, torch.int32), Buffer(np.array([len(self.free)], np.int32), torch.int32)
        self.kv = cp.PagedKV(pool, torch.zeros_like(pool), self.d_table.t[:, :cols])
        self.ctx = cp.Context(1, 1, 128, 1, 1, 1)

    def run(self, new, rows, in_place=False):
        n = len(self.have)
        d = [Buffer(np.asarray(x, np.int32), torch.int32) for x in (
            self.have, new, np.full(n, -3), np.full(n + 1, -3), np.full(rows, -3), np.full(rows, -3))]
        lens = d[0] if in_place else d[2]
        self.ctx.paged_plan(self.kv, d[0].t, d[1].t, self.d_free.t, self.d_count.t, lens.t, d[3].t, d[4].t, d[5].t)
        status = self.ctx.sync_status()
        want = oracle.plan_ref([int(h) for h in self.have], [int(x) for x in new], self.free, self.table, self.page, rows)
        # (the oracle's table has a column more than is in use)
        assert status == (cp.OK if want[4] else cp.E_PAGE)
        for got, w in zip((lens, d[3], d[4], d[5]), want):
            assert np.array_equal(got.host(), w)
        self.check()
        assert all(x.intact() for x in d)
        return want[0]

    def trim(self, lens, keep):
        d = [Buffer(np.asarray(x, np.int32), torch.int32) for x in (lens, keep)]
        self.ctx.paged_trim(self.kv, d[0].t, d[1].t, self.d_free.t, self.d_count.t)
        status = self.ctx.sync_status()
        oracle.trim_ref(lens, keep, self.free, self.table, self.page)
        self.check()
        return status

    def check(self):
        assert np.array_equal(self.d_table.host(), self.table)
        assert self.d_count.host()[0] == len(self.free)
        assert self.d_free.host()[:len(self.free)].tolist() == self.free
        assert self.d_table.intact() and self.d_free.intact() and self.d_count.intact()


RNG = np.random.default_rng(1)
PLANS = [  # have, new, page, spare pages, spare rows
    ([0], [1], 16, 1, 0), ([0], [0], 16, 0, 0), ([-1], [5], 16, 2, 3), ([15], [1], 16, 0, 1), ([16], [1], 16, 1, 0),
    ([500, 1, 16, 4095, 31, 777, 64], [1] * 7, 16, 9, 0),
    ([0, 5, -1, 0, 17], [300, 0, 9, 1, 40], 32, 100, 50),
    ([0, 0, 0], [9001, 1, 4096], 64, 300, 0),
    ([int(x) for x in RNG.integers(-1, 300, 1500)], [int(x) for x in RNG.integers(-2, 4, 1500)], 16, 2000, 7),
    ([int(x) for x in RNG.integers(0, 60, 4096)], [1] * 4096, 256, 5000, 0),
    ([0] * 40, [2000 + 13 * i for i in range(40)], 128, 800, 1000),
]


@pytest.mark.parametrize("in_place", [False, True], ids=["", "in_place"])
@pytest.mark.parametrize("have,new,page,spare,more", PLANS, ids=[f"{len(p[0])}x{p[2]}-{i}" for i, p in enumerate(PLANS)])
def test_plan_is_the_oracles_and_trim_undoes_it(have, new, page, spare, more, in_place):
    cols = max(1, max(-(-(h + max(n, 0)) // page) for h, n in zip(have, new) if h >= 0 or len(have) == 1)) + 2
    p = Plan(have, page, cols, spare)
    before, table = list(p.free), p.table.copy()
    rows = sum(max(n, 0) for h, n in zip(have, new) if h >= 0) + more
    lens = p.run(new, rows, in_place)
    assert p.trim(lens, have) == cp.OK
    assert p.free == before
    p.table[:], p.d_table = table, Buffer(table, torch.int32)
    # and all pages back
    p.kv = cp.PagedKV(p.kv.k_pages, p.kv.v_pages, p.d_table.t[:, :cols])
    assert p.trim(have, [0 if b % 3 else -1 for b in range(len(have))]) == cp.OK


def test_plan_serves_in_order_and_reports():
    """A list too short, a table row too short, rows past the call's: in order, and
    reported; a sequence that needs nothing is served all the same."""
    p = Plan([10, 16, 0, 30, -1, 5], 16, 4, 3)
    p.table = p.table[:, :4].copy()                   # the oracle's table has the columns in use
    p.d_table = Buffer(p.table, torch.int32)
    p.kv = cp.PagedKV(p.kv.k_pages, p.kv.v_pages, p.d_table.t)
    p.run([3, 17, 33, 2, 9, 0], 100)                  # b = 2 wants three pages, one is left
    p = Plan([10, 16, 0, 30, -1, 5], 16, 4, 20)
    p.table = p.table[:, :4].copy()
    p.d_table = Buffer(p.table, torch.int32)
    p.kv = cp.PagedKV(p.kv.k_pages, p.kv.v_pages, p.d_table.t)
    p.run([3, 49, 65, 2, 9, 0], 100)                  # b = 1 and 2 have more tokens than their rows of the table
    p = Plan([10, 16, 0, 30, -1, 5], 16, 4, 20)
    p.table = p.table[:, :4].copy()
    p.d_table = Buffer(p.table, torch.int32)
    p.kv = cp.PagedKV(p.kv.k_pages, p.kv.v_pages, p.d_table.t)
    p.run([3, 17, 5, 2, 9, 0], 22)                    # rows for the first two and a part of the third


def test_plan_of_no_rows_and_extreme_lengths():
    p = Plan([3, 7], 16, 2, 2)
    p.table = p.table[:, :2].copy()
    p.d_table = Buffer(p.table, torch.int32)
    p.kv = cp.PagedKV(p.kv.k_pages, p.kv.v_pages, p.d_table.t)
    p.run([0, 0], 0)
    d = [i32(x) for x in ([2 ** 31 - 1, 7], [2 ** 31 - 1, 2 ** 31 - 1], [0, 0], [0, 0, 0], [0] * 4, [0] * 4)]
    p.ctx.paged_plan(p.kv, d[0], d[1], p.d_free.t, p.d_count.t, d[2], d[3], d[4], d[5])
    assert p.ctx.sync_status() == cp.E_PAGE
    assert d[2].tolist() == [2 ** 31 - 1, 7] and d[4].tolist() == [-1] * 4 == d[5].tolist()
    assert d[3].tolist() == [0, 2 ** 31 - 1, 2 ** 31 - 1]       # (cut at int32's largest value)
    p.check()


def test_plan_reports_bad_pages_and_counts():
    p = Plan([0, 0], 16, 4, 4)
    p.d_free.t[3] = 10 ** 6                                    # the first page that goes
    d = [i32(x) for x in ([0, 0], [16, 16], [0, 0], [0, 0, 0], [0] * 32, [0] * 32)]
    p.ctx.paged_plan(p.kv, d[0], d[1], p.d_free.t, p.d_count.t, d[2], d[3], d[4], d[5])
    assert p.ctx.sync_status() == cp.E_PAGE
    assert d[5].tolist() == [-1] * 16 + [p.free[2] * 16 + i for i in range(16)]
    p.d_count.t[0] = 1000                                      # cut to the pool's four pages
    p.ctx.paged_plan(p.kv, d[0], i32([16, 0]), p.d_free.t, p.d_count.t, d[2], d[3], d[4], d[5])
    assert p.ctx.sync_status() == cp.E_PAGE and int(p.d_count.t[0]) == 3
    p.d_count.t[0] = -5
    p.ctx.paged_plan(p.kv, d[0], i32([1, 0]), p.d_free.t, p.d_count.t, d[2], d[3], d[4], d[5])
    assert p.ctx.sync_status() == cp.E_PAGE and int(p.d_count.t[0]) == 0 and d[2].tolist() == [0, 0]
    assert p.d_free.intact() and p.d_table.intact() and p.d_count.intact()


def test_trim_refuses_pages_twice_and_cuts_long_lengths():
    p = Plan([40, 20], 16, 3, 1)
    assert p.trim([40, 20], [0, -1]) == cp.OK
    before = list(p.free)
    p.ctx.paged_trim(p.kv, i32([40, 20]), i32([0, 0]), p.d_free.t, p.d_count.t)   # three pages a second time
    assert p.ctx.sync_status() == cp.E_PAGE
    p.free = before
    p.check()
    p.ctx.paged_trim(p.kv, i32([0, 10 ** 9]), i32([0, 32]), p.d_free.t, p.d_count.t)  # one column left of the table's
    assert p.ctx.sync_status() == cp.E_PAGE and int(p.d_count.t[0]) == len(before) + 1
    assert p.d_free.intact()


# --------------------------------------------------------- norm and rotation

# The bound of a value against float64, before its rounding: with |y_a| + |y_b| (or
# |y|) the sizes that enter it, fp32 makes of them
#   the norm: HD squares and their sum over lanes, (HD/32 + 13) roundings, halved by
#     the root, the root's 2 and the weight's 2:           <= 15 * 2^-24
#   the angle: 2^-25 half turns, so 2^-23.3; cos and sin 2 ulp: 2^-23; times scale: 2^-24
#   the two products and their sum:                        3 * 2^-24
# in all below 2^-19 of it.
def _bound(size):
    return 2.0 ** -19 * size + 1e-37


HEADS = [  # nq, nkv, hd, rows, rot, interleaved, weights, farthest position
    (1, 1, 128, 1, 128, False, "bf16", 10),
    (32, 2, 256, 7, 256, False, "bf16", 2 ** 20),
    (32, 4, 128, 130, 128, False, "f32", 2 ** 31 - 1),
    (7, 7, 128, 33, 64, True, "bf16", 100000),
    (3, 1, 256, 1000, 128, True, "f32", 2 ** 31 - 1),
    (16, 8, 128, 50, 24, False, "none", 4096),
    (6, 2, 256, 40, 8, True, "q", 4096),
    (5, 5, 256, 61, 104, False, "k", 9999),
    (8, 2, 128, 20, 0, False, "f32", 9999),
    (9, 3, 256, 20, 0, False, "none", 9999),
    (32, 2, 256, 3000, 256, False, "bf16", 5000),
]
IDS = [str(h) for h in HEADS]


def _randn(*shape):
    x = np.random.default_rng(sum(shape)).standard_normal(shape).astype(np.float32)
    return torch.from_numpy(x).to(torch.bfloat16).cuda()


class Heads:
    def __init__(self, nq, nkv, hd, rows, rot, interleaved, weights, far, seed=0, fused=True, pad=0):
        rng = np.random.default_rng(seed + hd + rows)
        self.freq = 5e5 ** (-np.arange(rot // 2) / max(rot // 2, 1))
        self.pos = rng.integers(0, far, rows).astype(np.int32)
        self.pos[:min(rows, 2)] = [0, far][:rows]
        wide = nq + 2 * nkv + pad
        x = rng.standard_normal((rows, wide, hd)) * 10.0 ** rng.integers(-3, 3, (rows, wide, 1))
        self.qkv = _bits(x)
        self.d_qkv = Buffer(self.qkv, torch.bfloat16)
        cut = (slice(0, nq), slice(nq, nq + nkv), slice(nq + nkv, nq + 2 * nkv))
        self.q, self.k, self.v = (self.qkv[:, c] for c in cut)
        self.d = [self.d_qkv.t[:, c] if fused else self.d_qkv.t[:, c].contiguous() for c in cut]
        w = [1 + 0.3 * rng.standard_normal(hd) for _ in range(2)]
        kind = torch.bfloat16 if weights != "f32" else torch.float32
        use = {"none": (0, 0), "q": (1, 0), "k": (0, 1)}.get(weights, (1, 1))
        d_w = [torch.from_numpy(x).to(kind).cuda() if u else None for x, u in zip(w, use)]
        self.w = [None if x is None else x.double().cpu().numpy() for x in d_w]
        self.eps, self.scale = 1e-5, 1.0
        self.kw = dict(eps=self.eps, interleaved=interleaved, scale=self.scale)
        self.nr = cp.NormRope(self.freq, *d_w, eps=self.eps, interleaved=interleaved)
        self.ctx = cp.Context(nq, nkv, hd, 1, 1, 1)
        self.d_pos = Buffer(self.pos, torch.int32)

    def ref(self, which):
        x = oracle.bits_to_f64((self.q, self.k)[which])
        return oracle.norm_rope_ref(x, self.pos, self.freq, self.w[which], **self.kw)


def _check_bf16(got, ref, size, skip=()):
    got = oracle.bits_to_f64(got)
    err, bound = np.abs(got - ref), 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -9) + _bound(size) * (1 + 2.0 ** -8)
    keep = np.setdiff1d(np.arange(len(ref)), skip)
    assert np.all(err[keep] <= bound[keep]), f"worst {np.max(err[keep] / bound[keep]):.3f} of the bound"


@pytest.mark.parametrize("fused", [True, False], ids=["fused", "dense"])
@pytest.mark.parametrize("case", HEADS, ids=IDS)
def test_norm_rope_parity(case, fused):
    h = Heads(*case, fused=fused)
    nq, nkv, hd, rows = case[:4]
    skip = [r for r in range(rows) if r % 11 == 5]
    h.d_pos.t[skip] = -1 - torch.arange(len(skip), dtype=torch.int32, device="cuda")
    out = [Buffer(np.full((rows, n, hd), 0x7FC1, np.uint16), torch.bfloat16) for n in (nq, nkv)]
    h.ctx.norm_rope(h.nr, h.d_pos.t, h.d[0], h.d[1], out[0].t, out[1].t)
    _ok(h.ctx)
    for i in range(2):
        ref, size = h.ref(i)
        _check_bf16(out[i].host(), ref, size, skip)
        assert np.all(out[i].host()[skip] == 0x7FC1) and out[i].intact()
    assert np.array_equal(h.d_qkv.host(), h.qkv) and h.d_qkv.intact()


@pytest.mark.parametrize("case", [HEADS[2], HEADS[3], HEADS[5], HEADS[9]], ids=str)
def test_norm_rope_in_place(case):
    """Within the projection's rows: the same bits as into other buffers, and V and the
    padding behind it are left alone."""
    h = Heads(*case, pad=3)
    nq, nkv, hd, rows = case[:4]
    out = [torch.zeros(rows, n, hd, dtype=torch.bfloat16, device="cuda") for n in (nq, nkv)]
    h.ctx.norm_rope(h.nr, h.d_pos.t, h.d[0], h.d[1], *out)
    h.ctx.norm_rope(h.nr, h.d_pos.t, h.d[0], h.d[1], h.d[0], h.d[1])
    _ok(h.ctx)
    assert torch.equal(h.d[0], out[0]) and torch.equal(h.d[1], out[1])
    assert np.array_equal(h.d_qkv.host()[:, nq + nkv:], h.qkv[:, nq + nkv:]) and h.d_qkv.intact()


def test_norm_rope_scale_and_extremes():
    """Rows of zeros, of the smallest and the largest values, and with a NaN or an
    infinity, which stays in its row and head; the rotated dims times a factor."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((8, 3, 128))
    x[1] = 0
    x[2] *= 1e-20                                   # (squares vanish against eps)
    x[3] *= 1e15
    bits = _bits(x)
    bits[4, 1, 7], bits[5, 0, 100] = 0x7FC1, 0xFF80
    t = Buffer(bits, torch.bfloat16)
    w = torch.from_numpy(1 + 0.1 * rng.standard_normal(128)).float().cuda()
    freq, pos = 1e4 ** (-np.arange(32) / 32), np.arange(8, dtype=np.int32) * 1000
    nr = cp.NormRope(freq, w, w, eps=1e-6, scale=1.25)
    ctx = cp.Context(3, 3, 128, 1, 1, 1)
    out = [Buffer(np.zeros_like(bits), torch.bfloat16) for _ in range(2)]
    ctx.norm_rope(nr, i32(pos), t.t, t.t, out[0].t, out[1].t)
    _ok(ctx)
    with np.errstate(invalid="ignore"):
        ref, size = oracle.norm_rope_ref(oracle.bits_to_f64(bits), pos, freq, w.double().cpu().numpy(), scale=1.25)
    got = oracle.bits_to_f64(out[0].host())
    assert np.array_equal(out[0].host(), out[1].host())
    bad = np.zeros((8, 3), bool)
    bad[4, 1] = bad[5, 0] = True
    assert np.isfinite(got[~bad]).all() and not np.isfinite(got[bad]).all(-1).any()
    assert np.all(np.abs(got - ref)[~bad] <= (2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -9) + _bound(size))[~bad])


# ------------------------------------------------------------------ append

APPENDS = [HEADS[0], HEADS[1], HEADS[2], HEADS[3], HEADS[4][:3] + (300,) + HEADS[4][4:], HEADS[5], HEADS[6], HEADS[7],
           HEADS[8], HEADS[9]]


def _spread(c, rows, seed):
    """Distinct slots of the pool for `rows` rows."""
    return np.random.default_rng(seed).choice(c.pools[0].shape[0] * c.page, rows, replace=False).astype(np.int32)


def _stored(c, slots):
    """Values [rows, NKV, HD] (float64) of K and V at the slots, and their scales."""
    at = slots // c.page, slice(None), slots % c.page
    pools = [d.host()[at] for d in c.d_pools]
    if c.scales is None:
        return [oracle.bits_to_f64(x) for x in pools], None
    recs = [d.host()[at] for d in c.d_scales]
    if c.scales[0].ndim == 4:
        return [oracle.values4(x, r) for x, r in zip(pools, recs)], recs
    return [oracle.e4m3_values()[x] * r[..., None].astype(np.float64) for x, r in zip(pools, recs)], recs


def _check_k(c, got, rec, ref, size):
    """K, quantised from fp32: within half a step of its stored scales, which follow from
    the largest values to fp32's accuracy."""
    err, off = np.abs(got - ref), _bound(size)
    if rec is None:
        assert np.all(err <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -9) + off * (1 + 2.0 ** -8))
    elif rec.ndim == 2:
        amax, loose = np.abs(ref).max(-1), off.max(-1)
        s = rec.astype(np.float64)
        assert np.all(np.abs(s * 448 - np.maximum(amax, 2.0 ** -110)) <= loose + 2.0 ** -22 * amax)
        half = np.maximum(2.0 ** -4 * (np.abs(ref) + off), s[..., None] * 2.0 ** -10)
        assert np.all(err <= half * (1 + 2.0 ** -20) + off)
    else:
        s = np.ascontiguousarray(rec[..., :4]).view(np.float32)[..., 0].astype(np.float64)
        r = oracle.e4m3_values()[rec[..., 4:]]
        amax, loose = np.abs(ref).max(-1), off.max(-1)
        assert np.all(np.exp2(np.round(np.log2(s))) == s)
        fine = amax > 2.0 ** -110
        assert np.all((s * 512 <= amax + loose)[fine]) and np.all((amax - loose < s * 1024))
        groups = lambda x: x.reshape(*x.shape[:-1], -1, 32)  # noqa: E731
        g, lo = np.abs(groups(ref)).max(-1), groups(off).max(-1)
        unit = s[..., None] * r
        assert np.all(np.abs(6 * unit - g) <= np.maximum(g / 16, 6 * s[..., None] * 2.0 ** -10) * (1 + 2.0 ** -20) + 2 * lo)
        u = np.repeat(unit, 32, -1)
        y = (np.abs(ref) + off) / np.where(u > 0, u, np.inf)
        half = np.where(y <= 2, .25, np.where(y <= 4, .5, 1.0)) * u * (1 + 2.0 ** -20)
        assert np.all(err <= np.where(u > 0, half, np.abs(ref)) + off)


@FORMATS
@pytest.mark.parametrize("case", APPENDS, ids=[str(a) for a in APPENDS])
def test_append_parity(case, fmt):
    h = Heads(*case)
    nq, nkv, hd, rows = case[:4]
    c = _paged(fmt, nkv, hd, 16, [rows + 40]).upload()
    slots = _spread(c, rows, rows)
    no_page = [r for r in range(rows) if r % 7 == 3]       # Q alone
    skip = [r for r in range(rows) if r % 11 == 5]         # nothing at all
    given = slots.copy()
    given[no_page] = -1
    h.d_pos.t[skip] = -1
    d_slots, out = Buffer(given, torch.int32), Buffer(np.full((rows, nq, hd), 0x7FC1, np.uint16), torch.bfloat16)
    before = [[d.host().copy() for d in x or []] for x in (c.d_pools, c.d_scales)]
    h.ctx.norm_rope_write_kv(h.nr, c.kv, h.d_pos.t, d_slots.t, *h.d, out.t)
    _ok(h.ctx)
    ref, size = h.ref(0)
    _check_bf16(out.host(), ref, size, skip)
    assert np.all(out.host()[skip] == 0x7FC1)
    assert out.intact() and c.intact() and d_slots.intact() and np.array_equal(h.d_qkv.host(), h.qkv)
    kept = np.setdiff1d(np.arange(rows), no_page + skip)
    vals, recs = _stored(c, slots[kept])
    ref, size = h.ref(1)
    if len(kept):
        _check_k(c, vals[0], None if recs is None else recs[0], ref[kept], size[kept])
    # V bit for bit, and nothing else of the pools touched
    at = slots[kept] // 16, slice(None), slots[kept] % 16
    for i in range(2):
        want = [x[i].copy() for x in before if x]
        if i == 0:
            for w, d in zip(want, [c.d_pools[0]] + ([c.d_scales[0]] if recs else [])):
                w[at] = d.host()[at]
        elif fmt == "bf16":
            want[0][at] = h.v[kept]
        elif fmt == "e4m3":
            want[0][at], want[1][at] = oracle.quantise_rows(h.v[kept])
        else:
            want[0][at], want[1][at] = oracle.quantise4_rows(oracle.bits_to_f64(h.v[kept]))
        for w, d in zip(want, [c.d_pools[i]] + ([c.d_scales[i]] if recs else [])):
            assert np.array_equal(w, d.host(), equal_nan=True)


@FORMATS
def test_append_without_norm_or_rotation_is_the_write(fmt):
    """K's bits are then paged_write_kv's."""
    nkv, hd, n = 3, 128, 50
    h = Heads(6, nkv, hd, n, 0, False, "none", 100)
    a, b = (_paged(fmt, nkv, hd, 32, [n], seed=5).upload() for _ in range(2))
    slots = [int(a.table[0, t // 32]) * 32 + t % 32 for t in range(n)]
    out = torch.zeros(n, 6, hd, dtype=torch.bfloat16, device="cuda")
    h.ctx.norm_rope_write_kv(h.nr, a.kv, h.d_pos.t, i32(slots), *h.d, out)
    h.ctx.paged_write_kv(b.kv, i32([0]), h.d[1].contiguous(), h.d[2].contiguous(), row_starts=i32([0, n]))
    _ok(h.ctx)
    for x, y in zip(a.d_pools + (a.d_scales or []), b.d_pools + (b.d_scales or [])):
        assert np.array_equal(x.host(), y.host(), equal_nan=True)
    assert torch.equal(out, h.d[0])


@FORMATS
def test_append_reports_slots_outside_the_pool_and_nan_rows(fmt):
    h = Heads(4, 2, 128, 4, 128, False, "bf16", 100)
    h.d_qkv.t[1, 4, 9] = float("nan")                       # row 1, K's first head
    c = _paged(fmt, 2, 128, 16, [64]).upload()
    before = [x.host().copy() for x in c.d_pools]
    out = torch.zeros(4, 4, 128, dtype=torch.bfloat16, device="cuda")
    last = c.pools[0].shape[0] * 16
    h.ctx.norm_rope_write_kv(h.nr, c.kv, h.d_pos.t, i32([last, 5, last - 1, 2 ** 31 - 1]), *h.d, out)
    assert h.ctx.sync_status() == cp.E_PAGE
    _ok(h.ctx)
    assert c.intact()
    vals, _ = _stored(c, np.array([5, last - 1]))
    assert np.isnan(vals[0][0, 0]).all() and np.isfinite(vals[0][0, 1]).all() and np.isfinite(vals[0][1]).all()
    assert np.isfinite(vals[1]).all()
    for x, d in zip(before, c.d_pools):
        changed = np.unique(np.argwhere(x != d.host())[:, [0, 2]] @ [16, 1])
        assert set(changed) <= {5, last - 1}


@pytest.mark.parametrize("nq,nkv,hd,rows,fmt", [(9, 1, 128, 7700, None), (2, 1, 256, 7400, None), (4, 2, 256, 7999, "e2m1"),
                                                (32, 2, 256, 7300, "bf16"), (6, 3, 128, 8000, "e4m3")], ids=str)
def test_many_rows_are_those_of_fewer_at_once(nq, nkv, hd, rows, fmt):
    """The same bits as calls of at most 2000 rows, which are dealt to the GPU in
    another way, with rows left out in both."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    qkv = torch.randn(rows, nq + 2 * nkv, hd, generator=gen, device="cuda").to(torch.bfloat16)
    x = qkv.split([nq, nkv, nkv], 1)
    pos = torch.randint(0, 2 ** 31 - 1, (rows,), generator=gen, device="cuda").int()
    pos[3::97] = -1
    w = torch.rand(hd, generator=gen, device="cuda") + 0.5
    nr = cp.NormRope(1e4 ** (-np.arange(hd // 2) / (hd // 2)), w, w)
    ctx = cp.Context(nq, nkv, hd, 1, 1, 1)
    slots = torch.randperm(rows, generator=gen, device="cuda").int()
    got = []
    for size in (rows, 2000):
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
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    ref, size = oracle.norm_rope_ref(x[0][-40:].double().cpu().numpy(), pos[-40:].tolist(),
                                     1e4 ** (-np.arange(hd // 2) / (hd // 2)), w.double().cpu().numpy())
    skip = np.flatnonzero(pos[-40:].cpu().numpy() < 0)
    _check_bf16(oracle.bf16_bits(got[0][0][-40:].cpu()), ref, size, skip)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_append_offsets_beyond_32_bits(fmt):
    """Rows 2^29 elements apart, and pools of more than 2^32 bytes whose last pages are used:
    the bits of a call on dense rows and a small pool."""
    nq, nkv, hd, rows, apart = 4, 2, 256, 6, 2 ** 29
    wide = nq + 2 * nkv
    far = torch.empty((rows - 1) * apart + wide * hd, dtype=torch.bfloat16, device="cuda")
    far = far.as_strided((rows, wide, hd), (apart, hd, 1))
    qkv = _randn(rows, wide, hd)
    far.copy_(qkv)
    pages, tail = (140000 if fmt == "e4m3" else 70000), 4
    dt = torch.float8_e4m3fn if fmt == "e4m3" else torch.bfloat16
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")

    def cache(n):
        pools = [torch.empty(n, nkv, 64, hd, dtype=dt, device="cuda") for _ in range(2)]
        scales = [torch.empty(n, nkv, 64, device="cuda") for _ in range(2)] if fmt == "e4m3" else []
        for x in pools + scales:
            x[-tail:].view(torch.uint8).zero_()
        return pools + scales, cp.PagedKV(*pools, table, *scales)

    nr = cp.NormRope(1e4 ** (-np.arange(128) / 128))
    ctx = cp.Context(nq, nkv, hd, 1, 1, 1)
    pos, at, got = i32([0, 5, 9, 70000, 2 ** 31 - 1, 3]), torch.tensor([255, 0, 77, 128, 9, 200]), []
    for x, n in ((qkv, tail), (far, pages)):
        held, kv = cache(n)
        q = torch.zeros(rows, nq, hd, dtype=torch.bfloat16, device="cuda")
        q = x[:, :nq] if n == pages else q                # (in place, far apart)
        ctx.norm_rope_write_kv(nr, kv, pos, i32((at + (n - tail) * 64).tolist()), *x.split([nq, nkv, nkv], 1), q)
        _ok(ctx)
        got.append([q.contiguous()] + [y[-tail:].contiguous().clone() for y in held])
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and a.view(torch.uint8).any()


# ------------------------------------------------------- the step as a whole

@FORMATS
@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
def test_steps_of_a_batch(fmt, captured):
    """Plan, append and attend, step after step: requests that grow over page borders,
    one that waits for a place, one that ends and another in its place; every step
    against the oracle over the cache as it stands."""
    rng = np.random.default_rng(21)
    nq, nkv, hd, page, B, cols = 8, 2, 128, 16, 4, 24
    c = _paged(fmt, nkv, hd, page, [page * 30])
    pages = c.pools[0].shape[0]
    c.table = np.full((B, cols), 2 ** 30, np.int32)
    c.cols = cols
    c.upload()
    ctx = cp.Context(nq, nkv, hd, 1, 1, 1)
    freq, w = 1e6 ** (-np.arange(64) / 64), [torch.ones(hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    nr = cp.NormRope(freq, *w)
    free, count = torch.randperm(pages, device="cuda", dtype=torch.int32), i32([pages])
    R = 4                                                    # rows of a decode step
    qkv = torch.zeros(R, nq + 2 * nkv, hd, dtype=torch.bfloat16, device="cuda")
    lens, new, starts, pos, slots = i32([0] * B), i32([0] * B), i32([0] * (B + 1)), i32([0] * R), i32([0] * R)
    q = torch.zeros(R, nq, hd, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros(B, nq, hd, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, nq, device="cuda")
    ws = torch.empty(ctx.paged_decode_workspace(B), dtype=torch.uint8, device="cuda")

    # prompts, of which the third place has none yet
    prompt = [37, 16, -1, 250]
    lens.copy_(i32(prompt).clamp_max(0))
    n = sum(max(x, 0) for x in prompt)
    big = torch.from_numpy(bf16_normal(rng, n, nq + 2 * nkv, hd).view(np.int16)).cuda().view(torch.bfloat16)
    p_pos, p_slots, p_q = i32([0] * n), i32([0] * n), torch.zeros(n, nq, hd, dtype=torch.bfloat16, device="cuda")
    ctx.paged_plan(c.kv, lens, i32(prompt), free, count, lens, starts, p_pos, p_slots)
    ctx.norm_rope_write_kv(nr, c.kv, p_pos, p_slots, *big.split([nq, nkv, nkv], 1), p_q)
    _ok(ctx)
    assert lens.tolist() == prompt and int(count) == pages - 3 - 1 - 16

    def step():
        ctx.paged_plan(c.kv, lens, new, free, count, lens, starts, pos, slots)
        ctx.norm_rope_write_kv(nr, c.kv, pos, slots, *qkv.split([nq, nkv, nkv], 1), q)
        ctx.paged_decode(c.kv, lens, q, out, ws, lse=lse)

    graph = None
    if captured:
        step_state = [x.clone() for x in (lens, free, count, c.d_table.t)]
        torch.cuda.synchronize()
        step()                                               # (kernels set up before the capture)
        torch.cuda.synchronize()
        for x, y in zip((lens, free, count, c.d_table.t), step_state):
            x.copy_(y)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    for i in range(5):
        if i == 2:                                           # a request ends, two come
            ctx.paged_trim(c.kv, lens, i32([-1, 0, -1, -1]), free, count)
            lens[1:3] = 0
        # (one row per place: an empty one's is behind the others')
        new.copy_((lens >= 0).int())
        host = bf16_normal(rng, R, nq + 2 * nkv, hd)
        qkv.copy_(torch.from_numpy(host.view(np.int16)).view(torch.bfloat16))
        before = lens.tolist()
        graph.replay() if captured else step()
        _ok(ctx)
        assert lens.tolist() == [x + 1 if x >= 0 else x for x in before]
        table = c.d_table.host()
        held = [table[b, :-(-max(x, 0) // page)] for b, x in enumerate(lens.tolist())]
        used = np.concatenate(held)
        assert len(set(used.tolist()) | set(free[:int(count)].tolist())) == pages == len(used) + int(count)
        # rows of this step: Q as the oracle turns it, and the attention over the pages
        rows = starts.tolist()
        c.pools = [d.host() for d in c.d_pools]
        c.scales = c.scales and [d.host() for d in c.d_scales]
        c.table = table
        for b, x in enumerate(before):
            if x >= 0:
                r = rows[b]
                assert int(pos[r]) == x
                ref, size = oracle.norm_rope_ref(oracle.bits_to_f64(host[r:r + 1, :nq]), [x], freq, np.ones(hd))
                _check_bf16(oracle.bf16_bits(q[r:r + 1].cpu()), ref, size)
        if min(before) < 0:
            # (rows are packed, the attention takes one per place)
            at = [rows[b] if x >= 0 else 3 for b, x in enumerate(before)]
            ctx.paged_decode(c.kv, lens, q[at].contiguous(), out, ws, lse=lse)
            _ok(ctx)
            d_q = oracle.bits_to_f64(oracle.bf16_bits(q[at].cpu()))
        else:
            d_q = oracle.bits_to_f64(oracle.bf16_bits(q.cpu()))
        got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        if fmt == "e2m1":
            check_decode4(c, d_q, lens.tolist(), hd ** -0.5, got, got_lse)
        else:
            ref = oracle.paged_decode_ref(d_q, c.pools, c.scales, c.table, page, lens.tolist(), hd ** -0.5)
            check_decode(got, got_lse, *ref, hd)


def test_prompts_are_normed_in_place_attended_and_kept():
    """Whole prompts: norm and rotation in place, packed attention, K and V written to
    4-bit pages, read back for a second turn."""
    rng = np.random.default_rng(22)
    nq, nkv, hd, lens = 8, 2, 128, [37, 1, 130]
    n = sum(lens)
    x = bf16_normal(rng, n, nq + 2 * nkv, hd)
    qkv = Buffer(x, torch.bfloat16)
    freq = 1e4 ** (-np.arange(64) / 64)
    nr = cp.NormRope(freq)
    ctx = cp.Context(nq, nkv, hd, 2, 100, 1)
    pos = np.concatenate([np.arange(k) for k in lens])
    q, k, v = (t.contiguous() for t in qkv.t.split([nq, nkv, nkv], 1))
    ctx.norm_rope(nr, i32(pos), q, k, q, k)
    out = torch.zeros_like(q)
    ws = torch.empty(ctx.prefill_packed_workspace(lens), dtype=torch.uint8, device="cuda")
    ctx.prefill_packed(lens, q, k, v, out, ws)
    c = Paged4(nkv, hd, 16, lens).upload()
    starts = np.concatenate([[0], np.cumsum(lens)])
    ctx.paged_write_kv(c.kv, i32([0, 0, 0]), k, v, row_starts=i32(starts))
    kc, vc = (torch.zeros(3, nkv, 2, 100, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ctx.paged_read_kv(c.kv, i32(lens), kc, vc)
    _ok(ctx)
    bits = [oracle.bf16_bits(t.cpu()) for t in (q, k, v)]
    ref, size = oracle.norm_rope_ref(oracle.bits_to_f64(x[:, :nq]), pos, freq)
    _check_bf16(bits[0], ref, size)
    oracle.paged_write_ref(c.pools, c.scales, c.table, 16, [0, 0, 0], starts, bits[1:])
    c.check_pools()
    for i, t in enumerate((kc, vc)):
        for b, m in enumerate(lens):
            want = oracle.paged_rows(c.pools[i], c.scales[i], c.table[b], 16, 0, m)
            tok = np.arange(m)
            assert np.array_equal(t[b].double().cpu().numpy()[:, tok % 2, tok // 2].swapaxes(0, 1), want)
    # the attention of the turned heads, last row of each prompt
    for b in range(3):
        rows = slice(starts[b], starts[b + 1])
        qq, kk, vv = (oracle.bits_to_f64(t)[rows] for t in bits)
        for h in range(nq):
            s = kk[:, h // 4] @ qq[-1, h] * hd ** -0.5
            p = np.exp(s - s.max())
            want = p @ vv[:, h // 4] / p.sum()
            got = out[starts[b + 1] - 1, h].double().cpu().numpy()
            assert np.abs(got - want).max() <= 2e-2


def test_two_streams_and_two_plans_at_once():
    """Two batches' steps on two streams, one context, own lists and tables."""
    ctx = cp.Context(2, 1, 128, 1, 1, 1)
    nr = cp.NormRope(1e4 ** (-np.arange(64) / 64))
    parts = []
    for s in range(2):
        p = Plan([20 + s, 0], 16, 12, 16, seed=s)
        new, rows = [100, 7 + s], 110
        d = [i32(x) for x in (p.have, new, [0, 0], [0, 0, 0], [0] * rows, [0] * rows)]
        x = torch.from_numpy(bf16_normal(np.random.default_rng(s), rows, 4, 128).view(np.int16)).cuda().view(torch.bfloat16)
        parts.append((p, new, rows, d, x, torch.zeros(rows, 2, 128, dtype=torch.bfloat16, device="cuda"),
                      torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for p, new, rows, d, x, q, st in parts:
            ctx.paged_plan(p.kv, d[0], d[1], p.d_free.t, p.d_count.t, d[2], d[3], d[4], d[5], stream=st)
            ctx.norm_rope_write_kv(nr, p.kv, d[4], d[5], *x.split([2, 1, 1], 1), q, stream=st)
            ctx.paged_trim(p.kv, d[2], d[0], p.d_free.t, p.d_count.t, stream=st)
    torch.cuda.synchronize()
    _ok(ctx)
    for p, new, rows, d, x, q, st in parts:
        before = list(p.free)
        lens, starts, pos, slots, fine = oracle.plan_ref([int(h) for h in p.have], new, p.free, p.table, 16, rows)
        assert fine and d[2].tolist() == lens and d[3].tolist() == starts
        assert np.array_equal(d[4].cpu().numpy(), pos) and np.array_equal(d[5].cpu().numpy(), slots)
        p.free = before
        p.check()
        n = starts[-1]
        ref, size = oracle.norm_rope_ref(x[:n, :2].double().cpu().numpy(), pos[:n], 1e4 ** (-np.arange(64) / 64))
        _check_bf16(oracle.bf16_bits(q[:n].cpu()), ref, size)


def test_binding_refuses_wrong_tensors():
    h = Heads(4, 2, 128, 3, 128, False, "bf16", 100)
    c = _paged("e4m3", 2, 128, 16, [64]).upload()
    out, ko = (torch.zeros(3, n, 128, dtype=torch.bfloat16, device="cuda") for n in (4, 2))
    good = dict(nr=h.nr, positions=h.d_pos.t, q=h.d[0], k=h.d[1], q_out=out, k_out=ko)
    for kw in (dict(positions=h.d_pos.t.long()), dict(positions=h.d_pos.t.cpu()), dict(q=h.d[0].float()),
               dict(q=h.d[0][:, :3]), dict(k=h.d[1].transpose(1, 2)), dict(k_out=ko[:2]), dict(q=h.d[0][..., ::2]),
               dict(q_out=out.cpu()), dict(positions=i32([1, 2]))):
        with pytest.raises(ValueError):
            h.ctx.norm_rope(**{**good, **kw})
    odd = torch.zeros(3 * 4 * 128 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(3, 4, 128)
    with pytest.raises(cp.CpattnError):
        h.ctx.norm_rope(**{**good, "q": odd})                 # not 16-byte aligned
    other = cp.Context(4, 2, 256, 1, 1, 1)
    with pytest.raises(ValueError):
        other.norm_rope(**good)
    with pytest.raises(ValueError):
        h.ctx.norm_rope_write_kv(h.nr, c.kv, h.d_pos.t, i32([1, 2]), *h.d, out)
    one = _randn(1, 4 * 128 + 4).as_strided((1, 4, 128), (4 * 128 + 4, 128, 1))
    h.ctx.norm_rope(h.nr, i32([1]), one, one[:, :2], out[:1], ko[:1])       # one row: its stride says nothing
    none = torch.zeros(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    h.ctx.norm_rope(h.nr, i32([]), none, none[:, :2], none, none[:, :2])    # no rows: nothing to do
    p = Plan([3], 16, 2, 2)
    args = [i32([3]), i32([1]), p.d_free.t, p.d_count.t, i32([0]), i32([0, 0]), i32([0]), i32([0])]
    for i in range(8):
        for bad in (args[i].long(), args[i].cpu(), torch.cat([args[i], args[i]])):
            if i == 6 and bad.numel() == 2:
                continue                                      # (then slots is the odd one out)
            with pytest.raises(ValueError):
                p.ctx.paged_plan(p.kv, *args[:i], bad, *args[i + 1:])
    for i in range(4):
        t = [i32([3]), i32([0]), p.d_free.t, p.d_count.t]
        t[i] = t[i].float()
        with pytest.raises(ValueError):
            p.ctx.paged_trim(p.kv, *t)
    p.check()
    _ok(h.ctx)
