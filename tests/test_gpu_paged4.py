"""4-bit pages on the GPU against the oracle: writes and reads bit for bit, decode
attention within a derived bound.  Every slot that no token was written to holds
ones in every bit, table columns behind a sequence name pages that do not exist,
and all buffers sit between canary bands."""
import numpy as np
import pytest
import torch

import long_context_chunked_gb300 as cp
import oracle
from long_context_chunked_gb300 import build as cpbuild
from long_context_chunked_gb300.binding import COUNT_BARS, COUNT_RECORD
from paged4_helpers import Paged4, check_decode4
from paged_helpers import Buffer, bf16_normal, i32
from test_gpu_paged import BRIEF, DECODES, READS, SPLITS, WRITES, _ok

pytestmark = pytest.mark.gpu


def _bits(x):
    return oracle.bf16_bits(torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16))


def _decode(c, nq, lens, seed=0, scale=0.0, q=None, ctx=None, with_lse=True, same_as=None):
    hd = c.hd
    if q is None:
        q = bf16_normal(np.random.default_rng(seed + 77), len(lens), nq, hd)
    d_q, d_out = Buffer(q, torch.bfloat16), Buffer(np.full(q.shape, 0x7FC1, np.uint16), torch.bfloat16)
    d_lse = Buffer(np.full(q.shape[:2], np.nan, np.float32), torch.float32)
    ctx = ctx or cp.Context(nq, c.nkv, hd, 1, 1, 1, scale)
    # the workspace starts as NaN: nothing of it may be used before it is written
    ws = Buffer(np.full(ctx.paged_decode_workspace(len(lens)), 0xFF, np.uint8), torch.uint8)
    ctx.paged_decode(c.kv, i32(lens), d_q.t, d_out.t, ws.t, lse=d_lse.t if with_lse else None)
    _ok(ctx)
    assert c.intact() and d_q.intact() and d_out.intact() and d_lse.intact() and ws.intact()
    if same_as:                              # (which was held against the oracle)
        assert np.array_equal(d_out.host(), same_as[0]) and np.array_equal(d_lse.host(), same_as[1])
        return same_as
    check_decode4(c, oracle.bits_to_f64(q), lens, scale or hd ** -0.5, oracle.bits_to_f64(d_out.host()),
                  d_lse.host().astype(np.float64) if with_lse else None)
    return d_out.host(), d_lse.host()


# ------------------------------------------------------------------ write and read

def _rows_of_all_kinds(rng, n, nkv, hd):
    """Rows over the whole range, groups of a row far apart, zeros, ties between codes,
    a row of subnormals and two rows without a scale."""
    f = rng.standard_normal((n, nkv, hd)) * 10.0 ** rng.integers(-37, 37, (n, nkv, 1))
    f *= 2.0 ** np.repeat(rng.integers(-20, 1, (n, nkv, hd // 32)), 32, -1)
    x = _bits(f)
    if n >= 8:
        ties = np.resize([6, .25, -.75, 1.25, 1.75, -2.5, 3.5, 5, .5, 0.0, -0.0], hd)
        x[0] = 0
        x[1] = _bits(ties * 3)
        x[2] = _bits(ties * 2.0 ** 100)
        x[3] = rng.integers(0, 128, (nkv, hd)).astype(np.uint16)        # subnormals
        x[4, 0, 5], x[5, nkv - 1, 7] = 0x7F80, 0xFFC1
        x[6] = 0x7F7F                                                  # the largest value of all
    return x


@pytest.mark.parametrize("nkv,hd,page,have,rows", WRITES, ids=[str(w[:3]) for w in WRITES])
def test_write_is_the_oracles(nkv, hd, page, have, rows):
    rng = np.random.default_rng(len(have) + nkv)
    c = Paged4(nkv, hd, page, [h + r for h, r in zip(have, rows)]).upload()
    lead, tail = 3, 2                        # rows of nobody before and behind
    starts = np.concatenate([[0], np.cumsum(rows)]) + lead
    new = [_rows_of_all_kinds(rng, starts[-1] + tail, nkv, hd) for _ in range(2)]
    d_new = [Buffer(x, torch.bfloat16) for x in new]
    ctx = cp.Context(nkv, nkv, hd, 1, 1, 1)
    ctx.paged_write_kv(c.kv, i32(have), d_new[0].t, d_new[1].t, row_starts=i32(starts))
    _ok(ctx)
    oracle.paged_write_ref(c.pools, c.scales, c.table, page, have, starts, new)
    c.check_pools()
    assert c.intact() and all(d.intact() for d in d_new)


def test_write_step_without_row_starts_and_skipped_sequences():
    rng = np.random.default_rng(8)
    have = [5, -1, 0, 47, -7, 16, 15, 31]
    c = Paged4(2, 128, 16, [max(h, 0) + 1 for h in have]).upload()
    new = [_rows_of_all_kinds(rng, 8, 2, 128) for _ in range(2)]
    ctx = cp.Context(4, 2, 128, 1, 1, 1)
    ctx.paged_write_kv(c.kv, i32(have), *(Buffer(x, torch.bfloat16).t for x in new))
    _ok(ctx)
    oracle.paged_write_ref(c.pools, c.scales, c.table, 16, have, np.arange(9), new)
    c.check_pools()
    assert c.intact()


@pytest.mark.parametrize("hd", [128, 256])
def test_write_step_of_the_largest_batches(hd):
    """One token each for so many sequences that a warp takes two of them."""
    rng = np.random.default_rng(10)
    have = [int(n) for n in rng.choice([-1, 0, 5, 15, 16, 31], cp.MAX_PAGED_SEQS - 3)]
    c = Paged4(3, hd, 16, [max(n, 0) + 1 for n in have]).upload()
    new = [bf16_normal(rng, len(have), 3, hd) for _ in range(2)]
    ctx = cp.Context(3, 3, hd, 1, 1, 1)
    ctx.paged_write_kv(c.kv, i32(have), *(Buffer(x, torch.bfloat16).t for x in new))
    _ok(ctx)
    oracle.paged_write_ref(c.pools, c.scales, c.table, 16, have, np.arange(len(have) + 1), new)
    c.check_pools()
    assert c.intact()


def test_write_beyond_the_table_and_bad_pages_are_reported():
    rng = np.random.default_rng(9)
    c = Paged4(2, 128, 16, [32, 32])
    c.table[1, 1] = -3
    c.upload()
    new = [bf16_normal(rng, 20, 2, 128) for _ in range(2)]
    d = [Buffer(x, torch.bfloat16).t for x in new]
    ctx = cp.Context(4, 2, 128, 1, 1, 1)
    ctx.paged_write_kv(c.kv, i32([25, 10]), *d, row_starts=i32([0, 10, 20]))
    assert ctx.sync_status() == cp.E_PAGE
    _ok(ctx)
    oracle.paged_write_ref(c.pools, c.scales, c.table, 16, [25], [0, 7], [x[:7] for x in new])
    oracle.paged_write_ref(c.pools, c.scales, c.table[1:], 16, [10], [0, 6], [x[10:16] for x in new])
    c.check_pools()
    assert c.intact()


@pytest.mark.parametrize("v_f16", [False, True], ids=["v_bf16", "v_f16"])
@pytest.mark.parametrize("nkv,hd,page,lens,P,S", READS, ids=[str(r[:3]) for r in READS])
def test_read_is_the_oracles(nkv, hd, page, lens, P, S, v_f16):
    rng = np.random.default_rng(P + nkv)
    c = Paged4(nkv, hd, page, lens)
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
            x = oracle.paged_rows(c.pools[i], c.scales[i], c.table[b], page, first[b], n)
            x = torch.from_numpy(x).to(torch.float16 if v_f16 and i else torch.bfloat16)
            for t in range(first[b], n):
                host[i][b, :, t % P, t // P] = x[t - first[b]].view(torch.int16).numpy().view(np.uint16)
        assert np.array_equal(d[i].host() & 0x7FFF, host[i] & 0x7FFF), "KV"[i]
        fine = (host[i] & 0x7FFF) != 0                # (zeros of either sign)
        assert np.array_equal(d[i].host()[fine], host[i][fine]), "KV"[i]
    assert all(x.intact() for x in d) and c.intact()


def test_read_reports_range():
    c = Paged4(2, 128, 16, [20])
    big = [np.full((1, 2, 128), 0x4780, np.uint16)] * 2  # 65536
    oracle.paged_write_ref(c.pools, c.scales, c.table, 16, [0], [0, 1], big)
    c.upload()
    ctx = cp.Context(2, 2, 128, 1, 32, 1, v_cache_f16=True)
    k, v = (torch.zeros(1, 2, 1, 32, 128, dtype=t, device="cuda") for t in (torch.bfloat16, torch.float16))
    ctx.paged_read_kv(c.kv, i32([1]), k, v)
    assert ctx.sync_status() == cp.E_RANGE
    assert torch.all(k[0, :, 0, 0] == 67584)       # s = 2^7, r = e4m3(512 / 6) = 88, 6 * 88 * 2^7


# ----------------------------------------------------------------- decode

@pytest.mark.parametrize("nq,nkv,hd,page,lens", DECODES, ids=[str(d[:4]) for d in DECODES])
def test_decode_parity(nq, nkv, hd, page, lens):
    c = Paged4(nkv, hd, page, lens, seed=nq)
    c.fill(np.random.default_rng(nq), lens)
    _decode(c.upload(), nq, lens)


@pytest.mark.parametrize("hd,page", [(128, 16), (256, 128)])
def test_decode_one_long_sequence_beside_short_ones(hd, page):
    lens = [1, 0, 40001, 2, 17]
    c = Paged4(2, hd, page, lens, seed=3)
    c.fill(np.random.default_rng(3), lens)
    _decode(c.upload(), 16, lens, with_lse=False)


def test_decode_many_sequences():
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.choice([0, 0, 1, 2, 16, 40, 90, 200], 700)]
    c = Paged4(2, 128, 16, lens, seed=4)
    c.fill(rng, lens)
    _decode(c.upload(), 4, lens)


@pytest.mark.parametrize("nq,nkv,hd,page,lens", SPLITS, ids=[f"{s[:4]}x{len(s[4])}" for s in SPLITS])
def test_decode_work_splits(nq, nkv, hd, page, lens):
    c = Paged4(nkv, hd, page, lens, seed=nq + hd)
    c.fill(np.random.default_rng(nq + hd), lens)
    c.upload()
    _decode(c, nq, lens, same_as=_decode(c, nq, lens))


@pytest.mark.parametrize("spare", [0, 4000])
@pytest.mark.parametrize("nq,nkv,hd,page,lens", [(b[0], b[1], b[2], b[3], [4 * n - n % 3 for n in b[4]]) for b in BRIEF],
                         ids=[f"{s[:4]}-{s[4][0]}" for s in BRIEF])
def test_decode_few_short_rows(nq, nkv, hd, page, lens, spare):
    """Around the longest rows that a CTA takes alone (twice as many tokens as of
    e4m3), with a table that ends behind them, and with one that could hold far more."""
    c = Paged4(nkv, hd, page, [n + spare for n in lens], seed=lens[0])
    c.fill(np.random.default_rng(lens[0]), lens)
    _decode(c.upload(), nq, lens)


def test_decode_of_the_largest_batch():
    rng = np.random.default_rng(16)
    B = cp.MAX_PAGED_SEQS
    lens = np.full(B, -1)
    used = rng.choice(B, 40, replace=False)
    lens[used] = rng.integers(1, 200, 40)
    lens[B - 1] = 133
    c = Paged4(1, 128, 16, np.maximum(lens, 0), seed=16)
    c.fill(rng, np.maximum(lens, 0))
    c.upload()
    out, _ = _decode(c, 2, [int(n) for n in lens])
    assert np.all(out[lens <= 0] == 0)


@pytest.mark.parametrize("q_scale", [2.0 ** -120, 2.0 ** 60, 30.0])
def test_decode_extreme_queries(q_scale):
    lens = [200, 3]
    c = Paged4(2, 128, 16, lens, seed=5)
    c.fill(np.random.default_rng(5), lens)
    c.upload()
    scale = 2.0 ** -60 / 128 ** 0.5 if q_scale > 1e6 else 0.0
    q = _bits(oracle.bits_to_f64(bf16_normal(np.random.default_rng(55), 2, 8, 128)) * q_scale)
    _decode(c, 8, lens, scale=scale, q=q)


@pytest.mark.parametrize("spread", [(30, 0), (0, 12), (20, 12)], ids=["tokens", "groups", "both"])
@pytest.mark.parametrize("nq,nkv,hd", [(8, 2, 128), (32, 2, 256)])
def test_decode_magnitudes_differ(nq, nkv, hd, spread):
    """V rows as far apart as 1e+-30, groups of a row as far as 2^-12 (K's as well)."""
    rng = np.random.default_rng(6)
    lens = [150, 33]
    c = Paged4(nkv, hd, 32, lens, seed=6)
    starts = np.concatenate([[0], np.cumsum(lens)])
    tokens, groups = spread
    new = []
    for i in range(2):
        f = rng.standard_normal((starts[-1], nkv, hd)) * 2.0 ** np.repeat(
            rng.integers(-groups, 1, (starts[-1], nkv, hd // 32)), 32, -1)
        new.append(_bits(f * 10.0 ** rng.integers(-tokens, tokens + 1, (starts[-1], nkv, 1)) if i else f))
    oracle.paged_write_ref(c.pools, c.scales, c.table, 32, [0, 0], starts, new)
    _decode(c.upload(), nq, lens)


def test_decode_takes_any_record():
    """Records that this library's writer does not make: every r_g up to 448, zero and
    subnormal ones among them, and s of any power of two."""
    rng = np.random.default_rng(7)
    lens = [300, 77]
    c = Paged4(2, 256, 64, lens, seed=7)
    c.fill(rng, lens)
    for i, (lo, hi) in enumerate([(-12, -8), (-60, 60)]):
        c.scales[i][..., 4:] = rng.integers(0, 0x7F, c.scales[i][..., 4:].shape)
        s = 2.0 ** rng.integers(lo, hi, c.scales[i].shape[:3])
        c.scales[i][..., :4] = s.astype(np.float32)[..., None].view(np.uint8)
        c.pools[i][...] = rng.integers(0, 256, c.pools[i].shape)
    _decode(c.upload(), 8, lens, scale=2.0 ** -8)


def test_decode_reports_bad_pages_and_lengths():
    lens = [140, 133, 120]
    c = Paged4(2, 128, 16, lens, seed=7)
    c.fill(np.random.default_rng(7), lens)
    c.table[1, 1] = 10 ** 6
    c.upload()
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, float("nan"))
    ctx = cp.Context(4, 2, 128, 1, 1, 1)
    ws = torch.empty(ctx.paged_decode_workspace(3), dtype=torch.uint8, device="cuda")
    ctx.paged_decode(c.kv, i32(lens), q, out, ws)
    assert ctx.sync_status() == cp.E_PAGE
    # q = 0: the mean of V, of the tokens whose page is there
    for b in range(3):
        v = oracle.paged_rows(c.pools[1], c.scales[1], np.where(c.table[b] < 10 ** 6, c.table[b], 0), 16, 0, lens[b])
        if b == 1:
            v = np.delete(v, np.s_[16:32], 0)
        got, mean = out[b, ::2].float().cpu().numpy(), v.mean(0)
        assert np.all(np.abs(got - mean) <= 2 ** -8 * np.abs(mean) + 2 ** -9.9 * np.abs(v).mean(0))
    _ok(ctx)
    ctx.paged_decode(c.kv, i32([140, 16, 10 ** 9]), q, out, ws)  # cut at the table's row, reported
    assert ctx.sync_status() == cp.E_PAGE
    ctx.paged_decode(c.kv, i32([40, -5, 20]), q, out, ws)
    _ok(ctx)
    assert torch.all(out[1] == 0) and c.intact()


def test_decode_nan_in_one_sequence_stays_there():
    rng = np.random.default_rng(11)
    lens = [50, 170, 130]
    c = Paged4(2, 128, 16, lens, seed=11)
    c.fill(rng, lens)
    bad = [np.full((1, 2, 128), 0x7FC1, np.uint16)] * 2
    oracle.paged_write_ref(c.pools, c.scales, c.table[1:], 16, [20], [0, 1], bad)
    c.upload()
    q = bf16_normal(rng, 3, 8, 128)
    out = torch.zeros(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    ctx = cp.Context(8, 2, 128, 1, 1, 1)
    ws = torch.empty(ctx.paged_decode_workspace(3), dtype=torch.uint8, device="cuda")
    ctx.paged_decode(c.kv, i32(lens), Buffer(q, torch.bfloat16).t, out, ws)
    _ok(ctx)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[[0, 2]]).all()
    c.table = c.table[[0, 2]]
    check_decode4(c, oracle.bits_to_f64(q[[0, 2]]), [50, 130], 128 ** -0.5, out[[0, 2]].double().cpu().numpy())


@pytest.mark.parametrize("nq,hd", [(8, 128), (16, 128), (8, 256), (16, 256)])
def test_slots_and_queries_reused_by_row_after_row(nq, hd):
    """Several rows for every warp, nearly all of which end inside a tile: the same
    bits every time, within the bound.  (All sequences share sixteen pages.)"""
    rng = np.random.default_rng(31)
    c = Paged4(1, hd, 16, [256], seed=31)
    c.fill(rng, [256])
    c.table = np.stack([rng.permutation(c.table[0, :16]) for _ in range(4000)]).astype(np.int32)
    c.upload()
    lens = [int(n) for n in rng.integers(1, 257, 4000)]
    _decode(c, nq, lens, same_as=_decode(c, nq, lens))


def test_offsets_beyond_32_bits():
    """Pools of more than 2^32 bytes whose last pages are used."""
    nkv, hd, page, pages = 2, 256, 64, 270000         # 4.4 GB of values for K and for V
    lens = [100, 64]
    kp = torch.empty(pages, nkv, page, hd // 2, dtype=torch.uint8, device="cuda")
    ks = torch.empty(pages, nkv, page, 4 + hd // 32, dtype=torch.uint8, device="cuda")
    vp, vs = torch.empty_like(kp), torch.empty_like(ks)
    table = np.array([[pages - 1, pages - 3], [pages - 2, 0]], np.int32)
    rng = np.random.default_rng(13)
    new = [bf16_normal(rng, 164, nkv, hd) for _ in range(2)]
    ctx = cp.Context(4, nkv, hd, 1, 128, 1)
    kv = cp.PagedKV(kp, vp, torch.from_numpy(table).cuda(), ks, vs)
    ctx.paged_write_kv(kv, i32([0, 0]), *(Buffer(x, torch.bfloat16).t for x in new), row_starts=i32([0, 100, 164]))
    q = bf16_normal(rng, 2, 4, hd)
    out, lse = torch.zeros(2, 4, hd, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 4, device="cuda")
    ws = torch.empty(ctx.paged_decode_workspace(2), dtype=torch.uint8, device="cuda")
    ctx.paged_decode(kv, i32(lens), Buffer(q, torch.bfloat16).t, out, ws, lse=lse)
    kc, vc = (torch.zeros(2, nkv, 1, 128, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ctx.paged_read_kv(kv, i32(lens), kc, vc)
    _ok(ctx)
    small = Paged4(nkv, hd, page, lens)
    small.table = np.array([[0, 1], [2, 3]], np.int32)
    oracle.paged_write_ref(small.pools, small.scales, small.table, page, [0, 0], [0, 100, 164], new)
    check_decode4(small, oracle.bits_to_f64(q), lens, hd ** -0.5, out.double().cpu().numpy(),
                  lse.double().cpu().numpy())
    for i, x in enumerate((kc, vc)):
        for b, n in enumerate(lens):
            want = oracle.paged_rows(small.pools[i], small.scales[i], small.table[b], page, 0, n)
            assert np.array_equal(x[b, :, 0, :n].transpose(0, 1).double().cpu().numpy(), want)


# ------------------------------------------------------- copies, waits

@pytest.fixture(scope="module")
def counted_lib():
    return cpbuild.build(variant="counted")


@pytest.mark.parametrize("drop", [False, True], ids=["healthy", "expired"])
@pytest.mark.parametrize("nq,nkv,hd,lens", [
    (8, 2, 128, [40001, 5]), (8, 2, 256, [20001, 5]), (16, 1, 256, [20001]), (8, 2, 128, [600]),
    (16, 1, 256, [300] * 350), (4, 4, 128, [1200 + 26 * i for i in range(40)])], ids=str)
def test_every_copy_lands_before_the_kernel_ends(counted_lib, nq, nkv, hd, lens, drop):
    """As tests/test_gpu_paged_edges.py has it for the other formats."""
    c = Paged4(nkv, hd, 64, lens, seed=33)
    if not drop:
        c.fill(np.random.default_rng(33), lens)
    c.upload()
    ctx = cp.Context(nq, nkv, hd, 1, 1, 1, library=counted_lib)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rec = torch.zeros(sms * COUNT_RECORD, dtype=torch.int32, device="cuda")
    ctx.set_barrier_counts(rec)
    q = torch.zeros(len(lens), nq, hd, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ctx.paged_decode_workspace(len(lens)), dtype=torch.uint8, device="cuda")
    if not drop:
        _decode(c, nq, lens, ctx=ctx)
    else:
        ctx.set_fault_injection(1, 50)
        ctx.paged_decode(c.kv, i32(lens), q, torch.zeros_like(q), ws)
        assert ctx.sync_status() == cp.E_TIMEOUT
    counts = rec.cpu().numpy().reshape(sms, -1, COUNT_BARS)
    assert np.array_equal(counts[:, 0], counts[:, 1])
    if drop:
        assert 0 < counts[0, 0, 0]
        ctx.set_fault_injection(0)
        rec.zero_()
        ctx.paged_decode(c.kv, i32(lens), q, torch.zeros_like(q), ws)
        assert ctx.sync_status() == cp.OK
        counts = rec.cpu().numpy().reshape(sms, -1, COUNT_BARS)
    # every tile's K and V once, in tiles of one size
    sent = int(counts[:, 0].sum())
    sizes = {2 * nkv * sum(-(-n // t) for n in lens) for t in (32, 64, 128)}
    assert sent in sizes and np.array_equal(counts[:, 0], counts[:, 1])


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
@pytest.mark.parametrize("hd,page", [(128, 16), (256, 64)])
def test_reads_between_writes_of_the_same_slots(hd, page, captured):
    rng = np.random.default_rng(35)
    nkv, n, turns = 2, 40, 12
    c = Paged4(nkv, hd, page, [n, n], seed=35).upload()
    ctx = cp.Context(nkv, nkv, hd, 1, n, 1)
    new = [[bf16_normal(rng, 2 * n, nkv, hd) for _ in range(2)] for _ in range(turns)]
    d_new = [[Buffer(x, torch.bfloat16).t for x in pair] for pair in new]
    got = torch.zeros(turns, 2, 2, nkv, 1, n, hd, dtype=torch.bfloat16, device="cuda")
    none, all_, starts = i32([0, 0]), i32([n, n]), i32([0, n, 2 * n])

    def chain():
        for (k, v), out in zip(d_new, got):
            ctx.paged_write_kv(c.kv, none, k, v, row_starts=starts)
            ctx.paged_read_kv(c.kv, all_, out[0], out[1])

    if captured:
        chain()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain()
        got.zero_()
        graph.replay()
    else:
        chain()
    _ok(ctx)
    for pair, out in zip(new, got.cpu()):
        oracle.paged_write_ref(c.pools, c.scales, c.table, page, [0, 0], [0, n, 2 * n], pair)
        for i in range(2):
            for b in range(2):
                want = oracle.paged_rows(c.pools[i], c.scales[i], c.table[b], page, 0, n)
                assert np.array_equal(out[i, b, :, 0].transpose(0, 1).double().numpy(), want)
    c.check_pools()


def test_binding_refuses_another_head_dim():
    c = Paged4(2, 128, 16, [20]).upload()
    q = torch.zeros(1, 4, 256, dtype=torch.bfloat16, device="cuda")
    ctx = cp.Context(4, 2, 256, 1, 1, 1)
    ws = torch.empty(ctx.paged_decode_workspace(1), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        ctx.paged_decode(c.kv, i32([3]), q, torch.zeros_like(q), ws)
