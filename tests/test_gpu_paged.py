"""The paged KV cache on the GPU against the oracle: writes and reads bit for
bit, decode attention within a derived bound.  Every slot that no token was
written to holds NaN, table columns behind a sequence name pages that do not
exist, and all buffers sit between canary bands."""
import numpy as np
import pytest
import torch

import long_context_chunked_gb300 as cp
import oracle
from paged_helpers import Buffer, Paged, bf16_normal, check_decode, i32

pytestmark = pytest.mark.gpu

FORMATS = pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])


def _ok(ctx):
    st = ctx.sync_status()
    assert st == cp.OK, f"status {st}: {ctx.last_error()}"


# ------------------------------------------------------------------ write

WRITES = [  # nkv, hd, page, cache lengths, new rows
    (1, 128, 16, [0], [1]),
    (2, 256, 16, [0, 15, 16, 17, 300], [1, 1, 1, 1, 1]),
    (4, 128, 64, [0, 63, 5, 100], [130, 2, 0, 1]),
    (3, 256, 32, [31, 0, 7], [33, 0, 1]),
    (8, 128, 256, [255, 1], [2, 700]),
    (5, 128, 128, [0] * 40, [37] * 40),      # several kv heads per warp
]


@FORMATS
@pytest.mark.parametrize("nkv,hd,page,have,rows", WRITES, ids=[str(w[:3]) for w in WRITES])
def test_write_is_the_oracles(nkv, hd, page, have, rows, e4m3):
    rng = np.random.default_rng(len(have) + nkv)
    c = Paged(nkv, hd, page, [h + r for h, r in zip(have, rows)], e4m3).upload()
    lead, tail = 3, 2                        # rows of nobody before and behind
    starts = np.concatenate([[0], np.cumsum(rows)]) + lead
    new = [bf16_normal(rng, starts[-1] + tail, nkv, hd) for _ in range(2)]
    if e4m3:  # magnitudes over the whole range, zeros, one row without a scale
        for x in new:
            f = oracle.bits_to_f64(x) * 10.0 ** rng.integers(-37, 37, x.shape[:2])[..., None]
            x[...] = oracle.bf16_bits(torch.from_numpy(f).to(torch.bfloat16))
            x[lead, 0] = 0
            x[starts[-1] - 1, 0, 5] = 0x7F80
    d_new = [Buffer(x, torch.bfloat16) for x in new]
    ctx = cp.Context(nkv, nkv, hd, 1, 1, 1)
    ctx.paged_write_kv(c.kv, i32(have), d_new[0].t, d_new[1].t, row_starts=i32(starts))
    _ok(ctx)
    oracle.paged_write_ref(c.pools, c.scales, c.table, page, have, starts, new)
    c.check_pools()
    assert c.intact() and all(d.intact() for d in d_new)


@FORMATS
def test_write_step_without_row_starts_and_skipped_sequences(e4m3):
    rng = np.random.default_rng(8)
    have = [5, -1, 0, 47, -7, 16]
    c = Paged(2, 128, 16, [max(h, 0) + 1 for h in have], e4m3).upload()
    new = [bf16_normal(rng, 6, 2, 128) for _ in range(2)]
    ctx = cp.Context(4, 2, 128, 1, 1, 1)
    ctx.paged_write_kv(c.kv, i32(have), *(Buffer(x, torch.bfloat16).t for x in new))
    _ok(ctx)
    oracle.paged_write_ref(c.pools, c.scales, c.table, 16, have, np.arange(7), new)
    c.check_pools()
    assert c.intact()


@FORMATS
def test_write_beyond_the_table_and_bad_pages_are_reported(e4m3):
    """Tokens behind the table's row, and a page id outside the pool: skipped,
    reported once, everything else written."""
    rng = np.random.default_rng(9)
    c = Paged(2, 128, 16, [32, 32], e4m3)
    c.table[1, 1] = -3
    c.upload()
    new = [bf16_normal(rng, 20, 2, 128) for _ in range(2)]
    d = [Buffer(x, torch.bfloat16).t for x in new]
    ctx = cp.Context(4, 2, 128, 1, 1, 1)
    ctx.paged_write_kv(c.kv, i32([25, 10]), *d, row_starts=i32([0, 10, 20]))
    assert ctx.sync_status() == cp.E_PAGE and "page" in ctx.last_error()
    _ok(ctx)  # the report is cleared
    # rows 0..6 fit the two pages of sequence 0, rows 10..15 the first page of sequence 1
    oracle.paged_write_ref(c.pools, c.scales, c.table, 16, [25], [0, 7], [x[:7] for x in new])
    oracle.paged_write_ref(c.pools, c.scales, c.table[1:], 16, [10], [0, 6], [x[10:16] for x in new])
    c.check_pools()
    ctx.paged_write_kv(c.kv, i32([2 ** 31 - 1, 10]), *d, row_starts=i32([0, 10, 10]))
    assert ctx.sync_status() == cp.E_PAGE
    c.check_pools()
    assert c.intact()


# ------------------------------------------------------------------- read

READS = [  # nkv, hd, page, lens, P, S
    (1, 128, 16, [1], 1, 1),
    (2, 256, 16, [0, 15, 16, 100], 3, 40),
    (4, 128, 64, [63, 65, 0, 300], 8, 38),
    (3, 256, 256, [257, 5], 2, 130),
    (8, 128, 32, [700] * 6, 1, 700),
]


@pytest.mark.parametrize("v_f16", [False, True], ids=["v_bf16", "v_f16"])
@FORMATS
@pytest.mark.parametrize("nkv,hd,page,lens,P,S", READS, ids=[str(r[:3]) for r in READS])
def test_read_is_the_oracles(nkv, hd, page, lens, P, S, e4m3, v_f16):
    rng = np.random.default_rng(P + nkv)
    c = Paged(nkv, hd, page, lens, e4m3)
    c.fill(rng, lens)
    c.upload()
    first = [n // 3 if b % 2 else 0 for b, n in enumerate(lens)]
    shape = (len(lens), nkv, P, S, hd)
    host = [rng.integers(0, 0x7B00, shape).astype(np.uint16) for _ in range(2)]
    d = [Buffer(host[0], torch.bfloat16), Buffer(host[1], torch.float16 if v_f16 else torch.bfloat16)]
    ctx = cp.Context(nkv, nkv, hd, P, S, 1, v_cache_f16=v_f16)
    ctx.paged_read_kv(c.kv, i32(lens), d[0].t, d[1].t, first=i32(first))
    _ok(ctx)
    for i in range(2):
        for b, n in enumerate(lens):
            x = oracle.paged_rows(c.pools[i], c.scales and c.scales[i], c.table[b], page, first[b], n)
            # an e4m3 value times an fp32 scale is rounded to fp32, then to the cache's type
            x = torch.from_numpy(x).float().to(torch.float16 if v_f16 and i else torch.bfloat16)
            for t in range(first[b], n):
                host[i][b, :, t % P, t // P] = x[t - first[b]].view(torch.int16).numpy().view(np.uint16)
        assert np.array_equal(d[i].host(), host[i]), "KV"[i]
    assert all(x.intact() for x in d) and c.intact()


@FORMATS
def test_read_cuts_long_lengths_and_reports_range(e4m3):
    rng = np.random.default_rng(5)
    c = Paged(2, 128, 16, [64, 64], e4m3)
    c.fill(rng, [64, 64])
    c.upload()
    shape = (2, 2, 2, 16, 128)       # 32 tokens fit
    d = [Buffer(np.full(shape, 0x1234, np.uint16), torch.bfloat16) for _ in range(2)]
    ctx = cp.Context(2, 2, 128, 2, 16, 1)
    ctx.paged_read_kv(c.kv, i32([64, 20]), d[0].t, d[1].t)
    assert ctx.sync_status() == cp.E_PAGE
    for i in range(2):
        for b, n in enumerate([32, 20]):
            x = torch.from_numpy(oracle.paged_rows(c.pools[i], c.scales and c.scales[i], c.table[b],
                                                   16, 0, n)).float().to(torch.bfloat16)
            got = d[i].t[b].cpu()
            for t in range(n):
                assert torch.equal(got[:, t % 2, t // 2], x[t])
        assert d[i].intact()
    assert np.all(d[0].host()[1, :, :, 10:] == 0x1234)
    # a V value beyond fp16's range, read into an fp16 cache
    big = [np.full((1, 2, 128), 0x4780, np.uint16), np.full((1, 2, 128), 0x4780, np.uint16)]  # 65536
    oracle.paged_write_ref(c.pools, c.scales, c.table, 16, [0], [0, 1], big)
    c.upload()
    ctx16 = cp.Context(2, 2, 128, 2, 16, 1, v_cache_f16=True)
    v16 = Buffer(np.zeros(shape, np.uint16), torch.float16)
    ctx16.paged_read_kv(c.kv, i32([20, 20]), d[0].t, v16.t)
    assert ctx16.sync_status() == cp.E_RANGE


# ----------------------------------------------------------------- decode

DECODES = [  # nq, nkv, hd, page, lens
    (1, 1, 128, 16, [1]),
    (2, 2, 256, 16, [0]),
    (8, 2, 128, 16, [1, 15, 16, 17, 31, 33, 0, 64, 65, 500]),
    (32, 2, 256, 64, [63, 1000, 0, 129]),
    (12, 4, 128, 256, [255, 256, 257, 2]),
    (6, 2, 256, 32, [0, 0, 95]),
    (32, 4, 128, 128, [700] * 12),
    (7, 7, 128, 16, [300, 3]),
    (20, 1, 128, 64, [1000, 127]),          # 20 q heads on one kv head
    (40, 1, 256, 16, [333]),
    (64, 2, 128, 32, [2000, 1]),
]


def _decode(c, nq, lens, seed=0, scale=0.0, q_scale=1.0, with_lse=True, ctx=None):
    rng = np.random.default_rng(seed + 77)
    hd = c.hd
    q = oracle.bits_to_f64(bf16_normal(rng, len(lens), nq, hd)) * q_scale
    q = oracle.bf16_bits(torch.from_numpy(q).to(torch.bfloat16))
    d_q, d_out = Buffer(q, torch.bfloat16), Buffer(np.full(q.shape, 0x7FC1, np.uint16), torch.bfloat16)
    d_lse = Buffer(np.full(q.shape[:2], np.nan, np.float32), torch.float32)
    ctx = ctx or cp.Context(nq, c.nkv, hd, 1, 1, 1, scale)
    # the workspace starts as NaN: nothing of it may be used before it is written
    ws = Buffer(np.full(ctx.paged_decode_workspace(len(lens)), 0xFF, np.uint8), torch.uint8)
    ctx.paged_decode(c.kv, i32(lens), d_q.t, d_out.t, ws.t, lse=d_lse.t if with_lse else None)
    _ok(ctx)
    assert c.intact() and d_q.intact() and d_out.intact() and d_lse.intact() and ws.intact()
    s = scale or hd ** -0.5
    ref = oracle.paged_decode_ref(oracle.bits_to_f64(q), c.pools, c.scales, c.table, c.page, lens, s)
    out = oracle.bits_to_f64(d_out.host())
    check_decode(out, d_lse.host().astype(np.float64) if with_lse else None, *ref, hd)
    if not with_lse:
        assert np.isnan(d_lse.host()).all()
    return d_out.host(), d_lse.host()


@FORMATS
@pytest.mark.parametrize("nq,nkv,hd,page,lens", DECODES, ids=[str(d[:4]) for d in DECODES])
def test_decode_parity(nq, nkv, hd, page, lens, e4m3):
    c = Paged(nkv, hd, page, lens, e4m3, seed=nq)
    c.fill(np.random.default_rng(nq), lens)
    _decode(c.upload(), nq, lens)


@FORMATS
@pytest.mark.parametrize("hd,page", [(128, 16), (256, 128)])
def test_decode_one_long_sequence_beside_short_ones(hd, page, e4m3):
    lens = [1, 0, 40001, 2, 17]
    c = Paged(2, hd, page, lens, e4m3, seed=3)
    c.fill(np.random.default_rng(3), lens)
    _decode(c.upload(), 16, lens, with_lse=False)


@FORMATS
def test_decode_many_sequences(e4m3):
    """More sequences than threads of a block, most of them empty or tiny."""
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.choice([0, 0, 1, 2, 16, 40, 90], 700)]
    c = Paged(2, 128, 16, lens, e4m3, seed=4)
    c.fill(rng, lens)
    _decode(c.upload(), 4, lens)


SPLITS = [  # nq, nkv, hd, page, lens: every way in which the rows share the GPU
    (16, 4, 128, 64, [5000, 7001, 6000, 8123, 4999, 9000, 100, 7777]),   # ends and beginnings in one CTA
    (32, 2, 256, 128, [3000, 4100, 2999, 3500, 0, 1, 6001, 2500]),
    (4, 2, 256, 32, [9001, 9001]),                                        # CTAs dealt evenly
    (16, 1, 256, 64, [20000]),
    (8, 4, 128, 32, [700 + 13 * i for i in range(60)]),                   # more rows than CTAs
    (32, 2, 256, 16, [1200, 900, 3] * 40),
    (8, 8, 128, 16, [2400, 2300, 2500, 2600] * 6),
    (4, 4, 256, 64, [1500, 20, 1700] * 20),
]


@FORMATS
@pytest.mark.parametrize("nq,nkv,hd,page,lens", SPLITS, ids=[f"{s[:4]}x{len(s[4])}" for s in SPLITS])
def test_decode_work_splits(nq, nkv, hd, page, lens, e4m3):
    c = Paged(nkv, hd, page, lens, e4m3, seed=nq + hd)
    c.fill(np.random.default_rng(nq + hd), lens)
    c.upload()
    a = _decode(c, nq, lens)
    b = _decode(c, nq, lens)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


BRIEF = [  # nq, nkv, hd, page, lens: around the longest rows that a CTA takes alone
    (8, 2, 128, 16, [768, 767, 1, 0]), (8, 2, 128, 16, [769, 3]),
    (8, 2, 128, 64, [1536, 1500]), (8, 2, 128, 64, [1537, 0]),
    (16, 1, 128, 32, [769]), (16, 1, 256, 32, [384, 383]), (16, 1, 256, 32, [385, 768]),
    (4, 2, 256, 16, [384, 5]), (4, 2, 256, 16, [577, 576]), (4, 2, 256, 16, [576, 0, 1]),
]


@FORMATS
@pytest.mark.parametrize("spare", [0, 2000])
@pytest.mark.parametrize("nq,nkv,hd,page,lens", BRIEF, ids=[f"{s[:4]}-{s[4][0]}" for s in BRIEF])
def test_decode_few_short_rows(nq, nkv, hd, page, lens, spare, e4m3):
    """With a table that ends behind them, and with one that could hold far more."""
    c = Paged(nkv, hd, page, [n + spare for n in lens], e4m3, seed=lens[0])
    c.fill(np.random.default_rng(lens[0]), lens)
    _decode(c.upload(), nq, lens)


@FORMATS
def test_decode_of_the_largest_batch(e4m3):
    """CPATTN_MAX_PAGED_SEQS sequences, most of them padding, some sharing pages."""
    rng = np.random.default_rng(16)
    B = cp.MAX_PAGED_SEQS
    lens = np.full(B, -1)
    used = rng.choice(B, 40, replace=False)
    lens[used] = rng.integers(1, 70, 40)
    lens[B - 1] = 33
    c = Paged(1, 128, 16, np.maximum(lens, 0), e4m3, seed=16)
    c.fill(rng, np.maximum(lens, 0))
    twin = int(used[0]) if used[0] != B - 1 else int(used[1])
    c.table[0], lens[0] = c.table[twin], lens[twin]       # a shared prefix
    c.upload()
    out, _ = _decode(c, 2, [int(n) for n in lens])
    assert np.all(out[lens <= 0] == 0)


@FORMATS
def test_decode_one_page_named_again_and_again(e4m3):
    """The longest sequence a table can name, every entry the same page: the
    page's own softmax, and an LSE that counts the copies.  Tokens are counted
    to less than a tile below 2^31.  A lane adds up 2^31 / (152 CTAs x 8 warps x
    8 lanes) = 2.2e5 probabilities at most in one fp32 sum, O as many products:
    each is off by at most 2.2e5 x 2^-24 = 1.4 % of A."""
    page, cols = 256, (1 << 31) // 256 - 1
    c = Paged(1, 128, page, [page], e4m3, seed=17)
    c.fill(np.random.default_rng(17), [page])
    c.upload()
    table = torch.full((1, cols), int(c.table[0, 0]), dtype=torch.int32, device="cuda")
    kv = cp.PagedKV(c.d_pools[0].t, c.d_pools[1].t, table,
                    *((s.t for s in c.d_scales) if e4m3 else (None, None)))
    q = bf16_normal(np.random.default_rng(18), 1, 4, 128)
    out = torch.zeros(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(1, 4, device="cuda")
    ctx = cp.Context(4, 1, 128, 1, 1, 1)
    ws = torch.empty(ctx.paged_decode_workspace(1), dtype=torch.uint8, device="cuda")
    ctx.paged_decode(kv, i32([2 ** 31 - 1]), Buffer(q, torch.bfloat16).t, out, ws, lse=lse)
    assert ctx.sync_status() == cp.E_PAGE                 # cut at the table's row
    ctx.paged_decode(kv, i32([cols * page]), Buffer(q, torch.bfloat16).t, out, ws, lse=lse)
    _ok(ctx)
    ref, ref_lse, A, X = oracle.paged_decode_ref(oracle.bits_to_f64(q), c.pools, c.scales, c.table, page,
                                                 [page], 128 ** -0.5)
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= 2 ** -8 * np.abs(ref) + 0.03 * A)
    assert np.all(np.abs(lse.double().cpu().numpy() - ref_lse - np.log(cols)) <= 0.02)


@FORMATS
@pytest.mark.parametrize("q_scale", [2.0 ** -120, 2.0 ** 60, 30.0])
def test_decode_extreme_queries(q_scale, e4m3):
    """Queries far below and above fp16's range (with a scale that brings the
    logits back to ordinary ones), and logits in the hundreds."""
    lens = [200, 3]
    c = Paged(2, 128, 16, lens, e4m3, seed=5)
    c.fill(np.random.default_rng(5), lens)
    c.upload()
    scale = 2.0 ** -60 / 128 ** 0.5 if q_scale > 1e6 else 0.0
    _decode(c, 8, lens, scale=scale, q_scale=q_scale)


@FORMATS
def test_decode_v_magnitudes_differ_by_token(e4m3):
    """V rows between 1e-30 and 1e30 (their e4m3 scales as far apart)."""
    rng = np.random.default_rng(6)
    lens = [150, 33]
    c = Paged(2, 128, 32, lens, e4m3, seed=6)
    starts = np.concatenate([[0], np.cumsum(lens)])
    new = [bf16_normal(rng, starts[-1], 2, 128) for _ in range(2)]
    f = oracle.bits_to_f64(new[1]) * 10.0 ** rng.integers(-30, 30, (starts[-1], 2, 1))
    new[1] = oracle.bf16_bits(torch.from_numpy(f).to(torch.bfloat16))
    oracle.paged_write_ref(c.pools, c.scales, c.table, 32, [0, 0], starts, new)
    _decode(c.upload(), 8, lens)


@FORMATS
def test_decode_reports_bad_pages_and_lengths(e4m3):
    lens = [40, 33, 20]
    c = Paged(2, 128, 16, lens, e4m3, seed=7)
    c.fill(np.random.default_rng(7), lens)
    c.table[1, 1] = 10 ** 6
    c.upload()
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, float("nan"))
    ctx = cp.Context(4, 2, 128, 1, 1, 1)
    ws = torch.empty(ctx.paged_decode_workspace(3), dtype=torch.uint8, device="cuda")
    ctx.paged_decode(c.kv, i32(lens), q, out, ws)
    assert ctx.sync_status() == cp.E_PAGE
    # q = 0: the mean of V; the other sequences are as ever
    for b in (0, 2):
        v = oracle.paged_rows(c.pools[1], c.scales and c.scales[1], c.table[b], 16, 0, lens[b])
        got = out[b, ::2].float().cpu().numpy()
        mean = v.mean(0)
        assert np.all(np.abs(got - mean) <= 2 ** -8 * np.abs(mean) + 2 ** -10 * np.abs(v).mean(0))
    assert torch.isfinite(out).all()
    _ok(ctx)
    c.table[1, 1] = c.table[0, 0]
    c.upload()
    ctx.paged_decode(c.kv, i32([40, 33, 10 ** 9]), q, out, ws)  # cut at the table's row, reported
    assert ctx.sync_status() == cp.E_PAGE
    ctx.paged_decode(c.kv, i32([40, -5, 20]), q, out, ws)
    _ok(ctx)
    assert torch.all(out[1] == 0)
    assert c.intact()


@FORMATS
def test_decode_nan_and_inf_in_one_sequence_stay_there(e4m3):
    """A sequence with a NaN token gives NaN; its neighbours do not."""
    rng = np.random.default_rng(11)
    lens = [50, 70, 30]
    c = Paged(2, 128, 16, lens, e4m3, seed=11)
    c.fill(rng, lens)
    bad = [np.full((1, 2, 128), 0x7FC1, np.uint16)] * 2
    oracle.paged_write_ref(c.pools, c.scales, c.table[1:], 16, [20], [0, 1], bad)
    c.upload()
    q = bf16_normal(rng, 3, 8, 128)
    d_q = Buffer(q, torch.bfloat16)
    out = torch.zeros(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    ctx = cp.Context(8, 2, 128, 1, 1, 1)
    ws = torch.empty(ctx.paged_decode_workspace(3), dtype=torch.uint8, device="cuda")
    ctx.paged_decode(c.kv, i32(lens), d_q.t, out, ws)
    _ok(ctx)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[[0, 2]]).all()
    ref = oracle.paged_decode_ref(oracle.bits_to_f64(q[[0, 2]]), c.pools, c.scales, c.table[[0, 2]],
                                  16, [50, 30], 128 ** -0.5)
    check_decode(out[[0, 2]].double().cpu().numpy(), None, *ref, 128)


@FORMATS
def test_decode_repeats_bit_for_bit(e4m3):
    lens = [1, 5000, 300, 0, 1234]
    c = Paged(2, 256, 32, lens, e4m3, seed=12)
    c.fill(np.random.default_rng(12), lens)
    c.upload()
    a = _decode(c, 32, lens)
    for _ in range(3):
        b = _decode(c, 32, lens)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes and 2^31 values whose last pages are used."""
    nkv, hd, page, pages = 2, 256, 64, 70000          # 2.3e9 values, 4.6 GB for K and for V
    lens = [100, 64]
    kp = torch.empty(pages, nkv, page, hd, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    table = np.array([[69999, 69997], [69998, 0]], np.int32)
    rng = np.random.default_rng(13)
    new = [bf16_normal(rng, 164, nkv, hd) for _ in range(2)]
    ctx = cp.Context(4, nkv, hd, 1, 128, 1)
    kv = cp.PagedKV(kp, vp, torch.from_numpy(table).cuda())
    d = [Buffer(x, torch.bfloat16).t for x in new]
    ctx.paged_write_kv(kv, i32([0, 0]), *d, row_starts=i32([0, 100, 164]))
    _ok(ctx)
    assert torch.equal(kp[69999, :, :64].transpose(0, 1), d[0][:64])
    q = bf16_normal(rng, 2, 4, hd)
    out, lse = torch.zeros(2, 4, hd, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 4, device="cuda")
    ws = torch.empty(ctx.paged_decode_workspace(2), dtype=torch.uint8, device="cuda")
    ctx.paged_decode(kv, i32(lens), Buffer(q, torch.bfloat16).t, out, ws, lse=lse)
    kc, vc = (torch.zeros(2, nkv, 1, 128, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ctx.paged_read_kv(kv, i32(lens), kc, vc)
    _ok(ctx)
    assert torch.equal(kc[0, :, 0, :100].transpose(0, 1), d[0][:100])
    assert torch.equal(vc[1, :, 0, :64].transpose(0, 1), d[1][100:])
    small = [np.zeros((4, nkv, page, hd), np.uint16) for _ in range(2)]
    tab = np.array([[0, 1], [2, 3]])
    oracle.paged_write_ref(small, None, tab, page, [0, 0], [0, 100, 164], new)
    ref = oracle.paged_decode_ref(oracle.bits_to_f64(q), small, None, tab, page, lens, hd ** -0.5)
    check_decode(out.double().cpu().numpy(), lse.double().cpu().numpy(), *ref, hd)


# ------------------------------------------------------- streams and graphs

@FORMATS
def test_captured_step_replays_with_new_lengths(e4m3):
    """One captured step (write the new token, attend) replayed while lengths
    and the table advance on the device."""
    rng = np.random.default_rng(14)
    nq, nkv, hd, page, B = 8, 2, 128, 16, 3
    have = np.array([14, 0, 63])
    steps = 4
    c = Paged(nkv, hd, page, list(have + steps), e4m3, seed=14)
    c.fill(rng, list(have))
    c.upload()
    ctx = cp.Context(nq, nkv, hd, 1, 1, 1)
    k, v = (torch.zeros(B, nkv, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B, nq, hd, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(B, nq, device="cuda")
    cached, lens = i32(have), i32(have + 1)
    ws = torch.empty(ctx.paged_decode_workspace(B), dtype=torch.uint8, device="cuda")

    def step():
        ctx.paged_write_kv(c.kv, cached, k, v)
        ctx.paged_decode(c.kv, lens, q, out, ws, lse=lse)

    def load(i):
        new = [bf16_normal(rng, B, nkv, hd) for _ in range(2)]
        qb = bf16_normal(rng, B, nq, hd)
        for t, x in ((k, new[0]), (v, new[1]), (q, qb)):
            t.copy_(torch.from_numpy(x.view(np.int16)).view(torch.bfloat16))
        oracle.paged_write_ref(c.pools, c.scales, c.table, page, list(have + i), np.arange(B + 1), new)
        return qb

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qb = load(0)
        step()                                   # warm-up is the first real step
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        if i:
            cached += 1
            lens += 1
            qb = load(i)
        graph.replay()                           # step 0 again: the same tokens, the same result
        _ok(ctx)
        c.check_pools()
        ref = oracle.paged_decode_ref(oracle.bits_to_f64(qb), c.pools, c.scales, c.table, page,
                                      list(have + i + 1), hd ** -0.5)
        check_decode(out.double().cpu().numpy(), lse.double().cpu().numpy(), *ref, hd)


def test_captured_forks_copies_and_shared_workspace():
    """A captured step whose decode follows a copy, then a fork of two streams,
    twice on one workspace; and an eager decode between its replays."""
    lens = [3000, 500, 17]
    ctx = cp.Context(16, 2, 128, 1, 1, 1)
    cs = [Paged(2, 128, 32, lens, bool(s), seed=50 + s) for s in range(2)]
    for s, c in enumerate(cs):
        c.fill(np.random.default_rng(50 + s), lens)
        c.upload()
    qs = [bf16_normal(np.random.default_rng(60 + s), 3, 16, 128) for s in range(2)]
    src = [Buffer(q, torch.bfloat16).t for q in qs]
    q = [torch.zeros_like(x) for x in src]
    out = [torch.zeros_like(x) for x in src]
    ws = [torch.empty(ctx.paged_decode_workspace(3), dtype=torch.uint8, device="cuda") for _ in range(2)]
    d_lens = i32([0] * 3)
    true_lens = i32(lens)
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        q[0].copy_(src[0], non_blocking=True)
        ctx.paged_decode(cs[0].kv, d_lens, q[0], out[0], ws[0])   # behind a copy
        side.wait_stream(here)
        with torch.cuda.stream(side):
            q[1].copy_(src[1])
            d_side.copy_(true_lens)
        here.wait_stream(side)
        ctx.paged_decode(cs[1].kv, d_side, q[1], out[1], ws[0])   # behind a join, same workspace

    d_side = i32([0] * 3)
    d_lens.copy_(true_lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    first = torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        ctx.paged_decode(cs[0].kv, d_lens, q[0], out[0], ws[0])   # the first node
    refs = [oracle.paged_decode_ref(oracle.bits_to_f64(x), c.pools, c.scales, c.table, 32, lens, 128 ** -0.5)
            for x, c in zip(qs, cs)]
    for _ in range(5):
        for t in out + q + [d_side]:
            t.zero_()
        graph.replay()
        ctx.paged_decode(cs[1].kv, true_lens, q[1], out[1], ws[0])
        got = [o.clone() for o in out]
        out[0].zero_()
        first.replay()
        _ok(ctx)
        for o, ref in ((got[0], refs[0]), (got[1], refs[1]), (out[0], refs[0])):
            check_decode(o.double().cpu().numpy(), None, *ref, 128)


def test_read_serves_shared_pages():
    """Two sequences whose tables name the same pages, read from odd places."""
    c = Paged(2, 128, 16, [50, 50], False, seed=70)
    c.fill(np.random.default_rng(70), [50, 50])
    c.table[1] = c.table[0]
    c.upload()
    ctx = cp.Context(2, 2, 128, 3, 17, 1)
    k, v = (torch.zeros(2, 2, 3, 17, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ctx.paged_read_kv(c.kv, i32([50, 50]), k, v, first=i32([1, 47]))
    _ok(ctx)
    for i, x in enumerate((k, v)):
        rows = torch.from_numpy(oracle.paged_rows(c.pools[i], None, c.table[0], 16, 0, 50)).to(torch.bfloat16)
        for b, first in enumerate((1, 47)):
            for t in range(51):
                want = rows[t] if first <= t < 50 else torch.zeros(2, 128, dtype=torch.bfloat16)
                assert torch.equal(x[b, :, t % 3, t // 3].cpu(), want), (i, b, t)


def test_two_streams_with_their_own_workspaces():
    """Two batches decoded on two streams at once, one context."""
    lens = [3000, 500, 17]
    ctx = cp.Context(16, 2, 128, 1, 1, 1)
    parts = []
    for s in range(2):
        c = Paged(2, 128, 32, lens, bool(s), seed=20 + s)
        c.fill(np.random.default_rng(20 + s), lens)
        c.upload()
        q = bf16_normal(np.random.default_rng(30 + s), 3, 16, 128)
        parts.append((c, q, Buffer(q, torch.bfloat16).t,
                      torch.zeros(3, 16, 128, dtype=torch.bfloat16, device="cuda"),
                      torch.empty(ctx.paged_decode_workspace(3), dtype=torch.uint8, device="cuda"),
                      torch.cuda.Stream()))
    d_lens = i32(lens)
    torch.cuda.synchronize()
    for _ in range(20):
        for c, q, d_q, out, ws, st in parts:
            ctx.paged_decode(c.kv, d_lens, d_q, out, ws, stream=st)
    torch.cuda.synchronize()
    _ok(ctx)
    for c, q, d_q, out, ws, st in parts:
        ref = oracle.paged_decode_ref(oracle.bits_to_f64(q), c.pools, c.scales, c.table, 32, lens, 128 ** -0.5)
        check_decode(out.double().cpu().numpy(), None, *ref, 128)


def test_binding_refuses_wrong_tensors():
    c = Paged(2, 128, 16, [20], False).upload()
    ctx = cp.Context(4, 2, 128, 1, 32, 1)
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ctx.paged_decode_workspace(1), dtype=torch.uint8, device="cuda")
    lens = i32([3])
    good = dict(pages=c.kv, lens=lens, q=q, out=torch.zeros_like(q), workspace=ws)
    for kw in (dict(q=q.float()), dict(q=q.transpose(1, 2)), dict(lens=lens.long()), dict(lens=i32([1, 2])),
               dict(out=torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")),
               dict(workspace=ws.cpu()), dict(lens=lens.cpu()), dict(lse=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            ctx.paged_decode(**{**good, **kw})
    with pytest.raises(cp.CpattnError):
        ctx.paged_decode(**{**good, "workspace": ws[:16]})
    other = cp.Context(4, 2, 256, 1, 1, 1)
    with pytest.raises(ValueError):
        other.paged_decode(**good)
    k = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(cp.CpattnError):
        ctx.paged_write_kv(c.kv, lens, k, k)          # two rows, one sequence, no row_starts
    with pytest.raises(ValueError):
        ctx.paged_write_kv(c.kv, lens, k, k[:1])
    with pytest.raises(ValueError):
        ctx.paged_read_kv(c.kv, lens, k, k)
    _ok(ctx)


@FORMATS
@pytest.mark.parametrize("hd", [128, 256])
def test_decode_wait_that_expires_is_reported(hd, e4m3):
    """A slot release skipped in the first CTA: its producer's wait runs into
    its limit, the kernel ends, the status says so, and the next call is right.
    (The first CTA must reuse its slots: two kv heads of 150000 tokens are
    2344 tiles of 128 or more, over 304 CTAs at least 7 each of two slots; the
    largest ring has 6.)"""
    lens = [150000, 5]
    c = Paged(2, hd, 64, lens, e4m3, seed=15)
    c.fill(np.random.default_rng(15), lens)
    c.upload()
    ctx = cp.Context(8, 2, hd, 1, 1, 1)
    q = torch.zeros(2, 8, hd, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ctx.paged_decode_workspace(2), dtype=torch.uint8, device="cuda")
    ctx.set_fault_injection(1, 50)
    ctx.paged_decode(c.kv, i32(lens), q, torch.zeros_like(q), ws)
    assert ctx.sync_status() == cp.E_TIMEOUT
    ctx.set_fault_injection(0)
    _decode(c, 8, lens, ctx=ctx)
