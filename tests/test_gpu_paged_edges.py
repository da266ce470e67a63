"""The paged decode where it can go wrong: slots and queries that are reused
row after row, copies in flight when a wait expires, V rows of very different
magnitudes, infinities.  Against the oracle, as tests/test_gpu_paged.py."""
import numpy as np
import pytest
import torch

import long_context_chunked_gb300 as cp
import oracle
from long_context_chunked_gb300 import build as cpbuild
from long_context_chunked_gb300.binding import COUNT_BARS, COUNT_RECORD
from paged_helpers import Buffer, Paged, bf16_normal, check_decode, i32
from test_gpu_paged import FORMATS, _decode, _ok

pytestmark = pytest.mark.gpu


@FORMATS
@pytest.mark.parametrize("nq,hd", [(8, 128), (16, 256)])
def test_slots_and_queries_reused_by_row_after_row(nq, hd, e4m3):
    """Several rows for every warp, nearly all of which end inside a tile: each
    warp clears the tail of a V slot, refills the slot and (16 heads of 256)
    takes the next row's Q into shared memory, again and again.  The same bits
    every time, within the bound.  (All sequences share eight pages.)"""
    rng = np.random.default_rng(31)
    c = Paged(1, hd, 16, [128], e4m3, seed=31)
    c.fill(rng, [128])
    c.table = np.stack([rng.permutation(c.table[0, :8]) for _ in range(4000)]).astype(np.int32)
    c.upload()
    lens = [int(n) for n in rng.integers(1, 129, 4000)]
    first = _decode(c, nq, lens)
    again = _decode(c, nq, lens)
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.fixture(scope="module")
def counted_lib():
    return cpbuild.build(variant="counted")


def _tile(hd, e4m3):
    """Tokens of a tile (DecodeLayout::WT)."""
    return 8192 // (hd * (1 if e4m3 else 2))


# nq, nkv, hd, lens.  The first slice of the list is long enough for a tile: the
# hook withholds the first copy of the first warp.
COPIES = [
    (8, 2, 128, [20001, 5]),             # a row that its whole CTA works on, cut across CTAs
    (8, 2, 256, [9001, 5]),
    (16, 1, 256, [9001]),                # the same, Q in shared memory
    (8, 2, 128, [300]),                  # a short row, alone in its CTA
    (16, 1, 256, [140] * 350),            # rows of its own, whole and cut
    (4, 4, 128, [600 + 13 * i for i in range(40)]),
]


@FORMATS
@pytest.mark.parametrize("drop", [False, True], ids=["healthy", "expired"])
@pytest.mark.parametrize("nq,nkv,hd,lens", COPIES, ids=[f"{s[:3]}x{len(s[3])}" for s in COPIES])
def test_every_copy_lands_before_the_kernel_ends(counted_lib, nq, nkv, hd, lens, drop, e4m3):
    """Every copy that a warp sends is seen to land, also where its first copy
    is withheld, so that its first wait runs into its limit with copies in
    flight behind it: the kernel then ends, the status says so, and the next
    call is right."""
    c = Paged(nkv, hd, 64, lens, e4m3, seed=33)
    if not drop:
        c.fill(np.random.default_rng(33), lens)
    c.upload()
    ctx = cp.Context(nq, nkv, hd, 1, 1, 1, library=counted_lib)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rec = torch.zeros(sms * COUNT_RECORD, dtype=torch.int32, device="cuda")
    ctx.set_barrier_counts(rec)
    tiles = sum(-(-n // _tile(hd, e4m3)) for n in lens) * nkv
    if not drop:
        _decode(c, nq, lens, ctx=ctx)
    else:
        ctx.set_fault_injection(1, 50)
        q = torch.zeros(len(lens), nq, hd, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(ctx.paged_decode_workspace(len(lens)), dtype=torch.uint8, device="cuda")
        ctx.paged_decode(c.kv, i32(lens), q, torch.zeros_like(q), ws)
        assert ctx.sync_status() == cp.E_TIMEOUT
    counts = rec.cpu().numpy().reshape(sms, -1, COUNT_BARS)
    sent, landed = counts[:, 0], counts[:, 1]
    assert np.array_equal(sent, landed)
    if not drop:
        assert sent.sum() == 2 * tiles
    else:
        assert 0 < sent[0, 0] and sent.sum() < 2 * tiles
        ctx.set_fault_injection(0)
        rec.zero_()
        ctx.paged_decode(c.kv, i32(lens), q, torch.zeros_like(q), ws)
        assert ctx.sync_status() == cp.OK
        counts = rec.cpu().numpy().reshape(sms, -1, COUNT_BARS)
        assert counts[:, 0].sum() == 2 * tiles and np.array_equal(counts[:, 0], counts[:, 1])


def test_counting_refuses_a_short_record(counted_lib):
    c = Paged(2, 128, 16, [4000] * 8, False, seed=34).upload()
    ctx = cp.Context(4, 2, 128, 1, 1, 1, library=counted_lib)
    ctx.set_barrier_counts(torch.zeros(COUNT_RECORD, dtype=torch.int32, device="cuda"))
    q = torch.zeros(8, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ctx.paged_decode_workspace(8), dtype=torch.uint8, device="cuda")
    with pytest.raises(cp.CpattnError):
        ctx.paged_decode(c.kv, i32([4000] * 8), q, torch.zeros_like(q), ws)


@FORMATS
@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
@pytest.mark.parametrize("hd,page", [(128, 16), (256, 64)])
def test_reads_between_writes_of_the_same_slots(hd, page, captured, e4m3):
    """Read, write, read, write .. of the same slots with nothing between the
    launches, each of which may start while the one ahead still runs: every
    read has the values (and scales) of the write before it."""
    rng = np.random.default_rng(35)
    nkv, n, turns = 2, 40, 12
    c = Paged(nkv, hd, page, [n, n], e4m3, seed=35).upload()
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
                want = oracle.paged_rows(c.pools[i], c.scales and c.scales[i], c.table[b], page, 0, n)
                want = torch.from_numpy(want).float().to(torch.bfloat16)
                assert torch.equal(out[i, b, :, 0].transpose(0, 1), want)
    c.check_pools()


def _bits(x):
    return oracle.bf16_bits(torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16))


# Which tokens of n differ, by which logit (the others' are within a few units
# of 0) and which factor of V.  The e4m3 scales of V differ as much: a token's
# scale may count only as far as its probability goes.
UNLIKE = {
    "first": lambda n, r: (np.arange(n) == 0, -50, 1e10),
    "last": lambda n, r: (np.arange(n) == n - 1, -50, 1e10),
    "middle": lambda n, r: (np.arange(n) == n // 2, -50, 1e10),
    "every 16th": lambda n, r: (np.arange(n) % 16 == 3, -50, 1e10),
    "every 2nd": lambda n, r: (np.arange(n) % 2 == 0, -60, 1e12),
    # one token has nearly all the probability and next to no V
    "sink": lambda n, r: (np.arange(n) == 0, 40, 1e-10),
    "late sink": lambda n, r: (np.arange(n) == n - 1, 40, 1e-10),
    # every product of a probability and a V is about as large as the others
    "balanced": lambda n, r: (np.ones(n, bool), (x := r.uniform(-30, 30, n)), np.exp(-x)),
}


@FORMATS
@pytest.mark.parametrize("where", UNLIKE)
@pytest.mark.parametrize("nq,nkv,hd,lens", [(8, 2, 128, [300, 40]), (32, 2, 256, [700, 33]), (4, 2, 256, [500]),
                                            (20, 1, 128, [5000])])
def test_v_magnitudes_against_probabilities(nq, nkv, hd, lens, where, e4m3):
    """Within check_decode's bound.  (P drops what is below 2^-31 of the largest
    product of a probability and a scale; here no product that A counts on is.)"""
    rng = np.random.default_rng(41)
    B = len(lens)
    base = rng.standard_normal((B, nkv, 1, hd))
    q = _bits((base + 0.02 * rng.standard_normal((B, nkv, nq // nkv, hd))).reshape(B, nq, hd))
    c = Paged(nkv, hd, 32, lens, e4m3, seed=41)
    starts = np.concatenate([[0], np.cumsum(lens)])
    k, v = (rng.standard_normal((starts[-1], nkv, hd)) for _ in range(2))
    for b, n in enumerate(lens):
        hit, logit, factor = UNLIKE[where](n, rng)
        at = starts[b] + np.flatnonzero(hit)
        unit = hd ** 0.5 * base[b, :, 0] / (base[b, :, 0] ** 2).sum(-1, keepdims=True)  # logit 1
        k[at] = np.broadcast_to(np.asarray(logit, float), n)[hit][:, None, None] * unit
        v[at] *= np.broadcast_to(np.asarray(factor, float), n)[hit][:, None, None]
    oracle.paged_write_ref(c.pools, c.scales, c.table, 32, [0] * B, starts, [_bits(k), _bits(v)])
    c.upload()
    out = torch.zeros(B, nq, hd, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(B, nq, device="cuda")
    ctx = cp.Context(nq, nkv, hd, 1, 1, 1)
    ws = torch.empty(ctx.paged_decode_workspace(B), dtype=torch.uint8, device="cuda")
    ctx.paged_decode(c.kv, i32(lens), Buffer(q, torch.bfloat16).t, out, ws, lse=lse)
    _ok(ctx)
    ref = oracle.paged_decode_ref(oracle.bits_to_f64(q), c.pools, c.scales, c.table, 32, lens, hd ** -0.5)
    check_decode(out.double().cpu().numpy(), lse.double().cpu().numpy(), *ref, hd)


@pytest.mark.parametrize("nq,nkv,hd,lens", [(8, 2, 128, [300, 40]), (32, 2, 256, [700, 33]), (4, 2, 256, [500]),
                                            (20, 1, 128, [170]), (16, 1, 128, [9000])])
def test_infinite_v_in_bf16_pages(nq, nkv, hd, lens):
    """+inf or -inf where a column of V has one (the first token, the last one,
    one between), NaN where it has both or a NaN; the other columns within the
    bound."""
    rng = np.random.default_rng(42)
    c = Paged(nkv, hd, 16, lens, False, seed=42)
    c.fill(rng, lens)
    for b, n in enumerate(lens):
        for t, d, x in ((0, 3, 0x7F80), (n - 1, 5, 0xFF80), (n // 4, 6, 0x7F80), (n // 2, 7, 0x7F80),
                        (n // 3, 7, 0xFF80), (n // 5, 9, 0x7FC1)):
            c.pools[1][c.table[b, t // 16], :, t % 16, d] = x
    c.upload()
    q = bf16_normal(rng, len(lens), nq, hd)
    out = torch.zeros(*q.shape, dtype=torch.bfloat16, device="cuda")
    ctx = cp.Context(nq, nkv, hd, 1, 1, 1)
    ws = torch.empty(ctx.paged_decode_workspace(len(lens)), dtype=torch.uint8, device="cuda")
    ctx.paged_decode(c.kv, i32(lens), Buffer(q, torch.bfloat16).t, out, ws)
    _ok(ctx)
    out = out.double().cpu().numpy()
    for d, want in ((3, np.inf), (5, -np.inf), (6, np.inf), (7, np.nan), (9, np.nan)):
        assert np.array_equal(out[..., d], np.full(out.shape[:2], want), equal_nan=True), d
    for b, n in enumerate(lens):
        for d in (3, 5, 6, 7, 9):
            c.pools[1][c.table[b, np.arange(n) // 16], :, np.arange(n) % 16, d] = 0
    keep = np.setdiff1d(np.arange(hd), (3, 5, 6, 7, 9))
    ref, lse, A, X = oracle.paged_decode_ref(oracle.bits_to_f64(q), c.pools, None, c.table, 16, lens, hd ** -0.5)
    check_decode(out[..., keep], None, ref[..., keep], lse, A[..., keep], X, hd)
