"""Packed prompts on the GPU against the oracle, and a whole request: prompt,
paged cache, decode steps, a second turn through the striped cache."""
import numpy as np
import pytest
import torch

import long_context_chunked_gb300 as cp
import oracle
from gpu_helpers import compare, to_f64
from paged_helpers import Buffer, Paged, bf16_normal, check_decode, i32

pytestmark = pytest.mark.gpu

CASES = [  # nq, nkv, hd, lens
    (1, 1, 128, [1]),
    (8, 2, 128, [37, 5, 128, 1, 64]),            # all short: GQA-packed
    (8, 2, 128, [300, 0, 129, 1, 0, 127, 128]),
    (4, 2, 256, [257, 64, 1000]),
    (3, 3, 128, [200, 131]),                     # no head pairs
    (12, 4, 256, [5, 700]),
    (16, 1, 128, [640]),
    (32, 4, 128, [513, 100] * 5),
    (2, 1, 256, [0, 0, 3]),
]


def _ref(q, k, v, lens, scale):
    out, lse, at = np.zeros(q.shape), np.zeros(q.shape[:2]), 0
    for n in lens:
        if n == 0:
            continue
        empty = np.zeros((1, k.shape[1], 1, 1, q.shape[2]))
        o, l = oracle.attend_ref(q[at:at + n], k[at:at + n], v[at:at + n], empty, empty, [0], [n], n, scale)
        out[at:at + n], lse[at:at + n] = o, l
        at += n
    return out, lse


def _run(nq, nkv, hd, lens, v_f16, pairing="mma2", poison=None, with_lse=True):
    rng = np.random.default_rng(sum(lens) + nq)
    T = sum(lens)
    bits = [bf16_normal(rng, T, h, hd) for h in (nq, nkv, nkv)]
    clean = [oracle.bits_to_f64(x) for x in bits]
    if poison is not None:                       # one sequence of NaN and infinities
        at = sum(lens[:poison])
        for x in bits:
            x[at:at + lens[poison]] = 0x7FC1
            x[at:at + lens[poison]:2] = 0xFF80
    d = [Buffer(x, torch.bfloat16) for x in bits]
    out = Buffer(np.full((T, nq, hd), 0x7F7F, np.uint16), torch.bfloat16)
    lse = Buffer(np.full((T, nq), 7e7, np.float32), torch.float32)
    ctx = cp.Context(nq, nkv, hd, 1, 1, 1, v_cache_f16=v_f16, pairing=pairing)
    ws = Buffer(np.full(ctx.prefill_packed_workspace(lens), 0xFF, np.uint8), torch.uint8)  # NaN
    ctx.prefill_packed(lens, d[0].t, d[1].t, d[2].t, out.t, ws.t, lse=lse.t if with_lse else None)
    st = ctx.sync_status()
    # (an infinity of the poisoned sequence lies outside fp16's range: reported)
    assert st == (cp.E_RANGE if poison is not None and v_f16 else cp.OK), ctx.last_error()
    assert all(b.intact() for b in (*d, out, lse, ws))
    ref, ref_lse = _ref(*clean, lens, hd ** -0.5)
    keep = np.ones(T, bool)
    if poison is not None:
        keep[at:at + lens[poison]] = False
    if keep.any():
        compare(to_f64(out.host())[keep], ref[keep], f"{nq}/{nkv} hd {hd} {lens}")
    if with_lse:
        assert np.max(np.abs(lse.host()[keep] - ref_lse[keep]), initial=0) < 2e-3
    else:
        assert np.all(lse.host() == np.float32(7e7))
    return out.host()


@pytest.mark.parametrize("v_f16", [False, True], ids=["v_bf16", "v_f16"])
@pytest.mark.parametrize("nq,nkv,hd,lens", CASES, ids=[str(c[:3]) for c in CASES])
def test_packed_parity(nq, nkv, hd, lens, v_f16):
    _run(nq, nkv, hd, lens, v_f16)


@pytest.mark.parametrize("pairing", ["none", "pingpong"])
def test_packed_other_kernel_forms(pairing):
    _run(8, 2, 128, [300, 0, 129, 1], True, pairing)
    _run(8, 2, 128, [300, 0, 129, 1], False, pairing, with_lse=False)


@pytest.mark.parametrize("v_f16", [False, True], ids=["v_bf16", "v_f16"])
@pytest.mark.parametrize("hd,lens", [(128, [100, 30, 77]), (256, [200, 333, 1]), (128, [20, 10, 7])],
                         ids=["128", "256", "short"])
def test_neighbours_of_a_nan_sequence_are_untouched(hd, lens, v_f16):
    for poison in range(3):
        _run(8, 2, hd, lens, v_f16, poison=poison)


def test_packed_equals_the_padded_prefill():
    """The same prompts through cpattn_prefill (padded rows, no cache): the
    same kernel on the same tiles gives the same bits."""
    rng = np.random.default_rng(1)
    lens, nq, nkv, hd, C = [300, 17, 128], 8, 2, 128, 320
    bits = [bf16_normal(rng, sum(lens), h, hd) for h in (nq, nkv, nkv)]
    t = [torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).cuda() for x in bits]
    ctx = cp.Context(nq, nkv, hd, 1, C, C, v_cache_f16=True)
    ws = torch.empty(ctx.prefill_packed_workspace(lens), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(t[0])
    ctx.prefill_packed(lens, *t, out, ws)
    pad = [torch.zeros(3 * C, x.shape[1], hd, dtype=torch.bfloat16, device="cuda") for x in t]
    at = 0
    for b, n in enumerate(lens):
        for p, x in zip(pad, t):
            p[b * C:b * C + n] = x[at:at + n]
        at += n
    stage = torch.empty(ctx.v_staging_bytes(3) // 2, dtype=torch.float16, device="cuda")
    ctx.set_v_staging(stage)
    kc = torch.zeros(3, nkv, 1, C, hd, dtype=torch.bfloat16, device="cuda")
    po = torch.zeros_like(pad[0])
    ctx.prefill([0, 0, 0], lens, *pad, kc, kc.half(), po)
    assert ctx.sync_status() == cp.OK
    at = 0
    for b, n in enumerate(lens):
        assert torch.equal(po[b * C:b * C + n], out[at:at + n])
        at += n


def test_packed_captured_twice_on_one_workspace():
    """Two captured graphs replayed one after the other share a workspace."""
    rng = np.random.default_rng(2)
    nq, nkv, hd = 8, 2, 128
    ctx = cp.Context(nq, nkv, hd, 1, 1, 1, v_cache_f16=True)
    batches = [[100, 200], [333]]
    ws = torch.empty(max(ctx.prefill_packed_workspace(x) for x in batches), dtype=torch.uint8, device="cuda")
    graphs = []
    for lens in batches:
        bits = [bf16_normal(rng, sum(lens), h, hd) for h in (nq, nkv, nkv)]
        t = [torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).cuda() for x in bits]
        out = torch.zeros_like(t[0])
        ctx.prefill_packed(lens, *t, out, ws)    # eager first: kernels are set up outside the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ctx.prefill_packed(lens, *t, out, ws)
        graphs.append((g, lens, bits, out, t))      # the graph reads t at every replay
    for _ in range(3):
        for g, lens, bits, out, _ in graphs:
            out.zero_()
            g.replay()
    assert ctx.sync_status() == cp.OK
    for g, lens, bits, out, _ in graphs:
        ref, _ = _ref(*(oracle.bits_to_f64(x) for x in bits), lens, hd ** -0.5)
        compare(out.double().cpu().numpy(), ref, str(lens))


# --------------------------------------------------------- a whole request

@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [128, 256])
def test_two_turns_of_a_batch(hd, e4m3):
    """Prompts are prefilled packed and written into pages; three decode steps
    append to them; a second turn reads the pages back into the striped cache
    and prefills a chunk on top, whose KV joins the pages too."""
    rng = np.random.default_rng(hd)
    nq, nkv, page, P = 8, 2, 32, 3
    lens = [150, 33, 1]
    B, steps, chunk = 3, 3, 70
    turn2 = [70, 0, 41]
    total = [a + steps + t for a, t in zip(lens, turn2)]
    S = -(-max(total) // P)
    scale = hd ** -0.5
    ctx = cp.Context(nq, nkv, hd, P, S, chunk, v_cache_f16=True)
    c = Paged(nkv, hd, page, total, e4m3, seed=hd).upload()
    # turn 1: the prompts
    q, k, v = (bf16_normal(rng, sum(lens), h, hd) for h in (nq, nkv, nkv))
    d = [Buffer(x, torch.bfloat16).t for x in (q, k, v)]
    ws = torch.empty(ctx.prefill_packed_workspace(lens), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(d[0])
    ctx.prefill_packed(lens, *d, out, ws)
    starts = np.concatenate([[0], np.cumsum(lens)])
    ctx.paged_write_kv(c.kv, i32([0] * B), d[1], d[2], row_starts=i32(starts))
    ref, _ = _ref(*(oracle.bits_to_f64(x) for x in (q, k, v)), lens, scale)
    assert ctx.sync_status() == cp.OK
    compare(out.double().cpu().numpy(), ref, "prompt")
    oracle.paged_write_ref(c.pools, c.scales, c.table, page, [0] * B, starts, [k, v])
    # decode steps
    dws = torch.empty(ctx.paged_decode_workspace(B), dtype=torch.uint8, device="cuda")
    for i in range(steps):
        q, k, v = (bf16_normal(rng, B, h, hd) for h in (nq, nkv, nkv))
        d = [Buffer(x, torch.bfloat16).t for x in (q, k, v)]
        have = [n + i for n in lens]
        ctx.paged_write_kv(c.kv, i32(have), d[1], d[2])
        out = torch.zeros_like(d[0])
        ctx.paged_decode(c.kv, i32([n + 1 for n in have]), d[0], out, dws)
        assert ctx.sync_status() == cp.OK
        oracle.paged_write_ref(c.pools, c.scales, c.table, page, have, np.arange(B + 1), [k, v])
        r = oracle.paged_decode_ref(oracle.bits_to_f64(q), c.pools, c.scales, c.table, page,
                                    [n + 1 for n in have], scale)
        check_decode(out.double().cpu().numpy(), None, *r, hd)
    c.check_pools()
    # turn 2: the pages' values in the striped cache, a chunk on top
    have = [n + steps for n in lens]
    kc = torch.zeros(B, nkv, P, S, hd, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros(B, nkv, P, S, hd, dtype=torch.float16, device="cuda")
    ctx.paged_read_kv(c.kv, i32(have), kc, vc)
    T = B * chunk
    q, k, v = (bf16_normal(rng, T, h, hd) for h in (nq, nkv, nkv))
    d = [Buffer(x, torch.bfloat16).t for x in (q, k, v)]
    out = torch.zeros_like(d[0])
    ctx.prefill(have, turn2, *d, kc, vc, out)
    pad_starts = [b * chunk for b in range(B)]
    rows = [np.concatenate([np.arange(s, s + n) for s, n in zip(pad_starts, turn2)])]
    packed = [torch.from_numpy(x[rows[0]].view(np.int16)).view(torch.bfloat16).cuda() for x in (k, v)]
    s2 = np.concatenate([[0], np.cumsum(turn2)])
    ctx.paged_write_kv(c.kv, i32(have), *packed, row_starts=i32(s2))
    assert ctx.sync_status() == cp.OK
    oracle.paged_write_ref(c.pools, c.scales, c.table, page, have, s2, [k[rows[0]], v[rows[0]]])
    c.check_pools()
    ref, _ = oracle.attend_ref(*(oracle.bits_to_f64(x) for x in (q, k, v)),
                               kc.double().cpu().numpy(), vc.double().cpu().numpy(), have, turn2,
                               chunk, scale)
    got = out.double().cpu().numpy()
    for b, n in enumerate(turn2):
        if n:
            compare(got[b * chunk:b * chunk + n], ref[b * chunk:b * chunk + n], f"turn 2, sequence {b}")
    assert c.intact()
