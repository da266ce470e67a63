"""Edges of attention over 4-bit pages on the GPU: column groups that are small in
every token, next to a token that outweighs the others; values next to the largest;
and the number of copies, in tiles of the one size that each kernel has."""
import numpy as np
import pytest
import torch

import long_context_chunked_gb300 as cp
import oracle
from long_context_chunked_gb300 import build as cpbuild
from long_context_chunked_gb300.binding import COUNT_BARS, COUNT_RECORD
from paged4_helpers import Paged4, largest_product
from paged_helpers import Buffer, i32
from test_gpu_paged import _ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("small", [-6, -9])
@pytest.mark.parametrize("nq,hd", [(8, 128), (16, 128), (8, 256), (16, 256)])
def test_small_groups_keep_their_tokens(nq, hd, small):
    """One token has 2^17.4 times the others' probability and nothing in the second group of V,
    where every other token has r_g = 2^small (2^7 in the other groups): the group's output
    is the others' alone, and is held to a bound of its own size.  Each warp has a whole
    sequence or most of it, so that the large product is the reference of its tokens.

    Of the bound: P = p s 2^7 / W, W at most twice M, the largest p s, is rounded once to
    fp16: 2^-11 of it, or in fp16's subnormals half of 2^-24; a token's value is at most
    6 s r_g and O's unit W / 2^7, so that is 2^-25 * 6 r_g * 2 M / 2^7 = 12 r_g M 2^-32 for
    every token.  r_g x4 has 6 significant bits: no rounding.  The logits' error and fp32 as
    in out_bound."""
    rng = np.random.default_rng(hd + nq)
    n, page, seqs = 1500, 64, 2048
    c = Paged4(1, hd, page, [n])
    for pool, scale in zip(c.pools, c.scales):
        pool[...] = rng.integers(0, 256, pool.shape) & 0x77        # codes without a sign
        scale[..., :4] = np.array([1.0], np.float32).view(np.uint8)
        scale[..., 4:] = 0x70                                      # 2^7
    c.scales[1][..., 5] = 0x08 if small == -6 else 0x01            # 2^-6, 2^-9
    # K is 0 but for the large token's first value, q is 1 there
    c.pools[0][...] = 0
    big = c.table[0, 700 // page], 0, 700 % page
    c.pools[0][big][0] = 0x02                                      # 1
    c.pools[1][big][16:32] = 0
    q = np.zeros((1, nq, hd), np.float32)
    q[..., 0] = 1
    scale = 17.4 * np.log(2) / 2 ** 7                              # (the token's logit: 17.4 ln 2)
    c.table = np.repeat(c.table, seqs, 0)
    c.upload()
    ctx = cp.Context(nq, 1, hd, 1, 1, 1, scale)
    bits = oracle.bf16_bits(torch.from_numpy(np.repeat(q, seqs, 0)).to(torch.bfloat16))
    d_q, out = Buffer(bits, torch.bfloat16), torch.zeros(seqs, nq, hd, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ctx.paged_decode_workspace(seqs), dtype=torch.uint8, device="cuda")
    ctx.paged_decode(c.kv, i32([n] * seqs), d_q.t, out, ws)
    _ok(ctx)
    assert c.intact()
    c.table = c.table[:1]
    s32 = float(np.float32(scale))
    ref, _, A, X = oracle.paged_decode_ref(q.astype(np.float64), c.pools, c.scales, c.table, page, [n], s32)
    M = largest_product(q.astype(np.float64), c, [n], s32)[..., None]
    r = np.full(hd, 2.0 ** 7)
    r[32:64] = 2.0 ** small
    bound = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -9) + A * (2.0 ** -11 + 2 * hd * 2.0 ** -23 * X[..., None] + 2.0 ** -20) \
        + n * 12 * 2.0 ** -32 * r * M
    got = out.double().cpu().numpy()
    err = np.abs(got - ref)
    assert np.all(err <= bound), f"worst {np.max(err / bound):.3f} of the bound"


@pytest.mark.parametrize("hd", [128, 256])
def test_values_next_to_the_largest(hd):
    """A row whose largest value is above 1008 * 2^118 has r_g = 176, and its values above 5
    * 176 * 2^118 read back as 6 * 176 * 2^118: an infinity.  From 1008 * 2^118 down: 160."""
    x = np.zeros((2, 1, hd))
    x[0, 0, :3] = np.array([1012, 884, -876]) * 2.0 ** 118
    x[1, 0, :3] = np.array([1008, -884, 700]) * 2.0 ** 118
    bits = oracle.bf16_bits(torch.from_numpy(x).to(torch.bfloat16))
    assert np.array_equal(oracle.bits_to_f64(bits), x)
    c = Paged4(1, hd, 16, [2]).upload()
    ctx = cp.Context(1, 1, hd, 1, 2, 1)
    d = [Buffer(bits, torch.bfloat16).t for _ in range(2)]
    ctx.paged_write_kv(c.kv, i32([0]), *d, row_starts=i32([0, 2]))
    cache = [torch.zeros(1, 1, 1, 2, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ctx.paged_read_kv(c.kv, i32([2]), *cache)
    _ok(ctx)
    for y in cache:
        y = y[0, 0, 0].double().cpu().numpy()
        assert y[0, :3].tolist() == [np.inf, np.inf, -704 * 2.0 ** 118] and not y[:, 3:].any()
        assert y[1, :3].tolist() == [960 * 2.0 ** 118, -960 * 2.0 ** 118, 640 * 2.0 ** 118]


@pytest.mark.parametrize("nq,nkv,hd,page,lens", [
    (8, 2, 128, 64, [40001, 5]), (16, 1, 128, 16, [20001, 300]), (8, 2, 256, 64, [20001, 5]), (16, 1, 256, 128, [20001]),
    (16, 1, 256, 64, [300] * 350), (8, 1, 256, 16, [33 + i for i in range(300)]), (4, 4, 128, 32, [1200 + 26 * i for i in range(40)])],
    ids=str)
def test_every_tile_is_copied_once(nq, nkv, hd, page, lens):
    """K and V of each tile: of 32 tokens for more than 8 heads of 256 to a kv head, else of 64."""
    c = Paged4(nkv, hd, page, lens, seed=33)
    c.fill(np.random.default_rng(33), lens)
    c.upload()
    ctx = cp.Context(nq, nkv, hd, 1, 1, 1, library=cpbuild.build(variant="counted"))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rec = torch.zeros(sms * COUNT_RECORD, dtype=torch.int32, device="cuda")
    ctx.set_barrier_counts(rec)
    q = torch.zeros(len(lens), nq, hd, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ctx.paged_decode_workspace(len(lens)), dtype=torch.uint8, device="cuda")
    ctx.paged_decode(c.kv, i32(lens), q, torch.zeros_like(q), ws)
    _ok(ctx)
    tile = 32 if hd == 256 and nq // nkv > 8 else 64
    counts = rec.cpu().numpy().reshape(sms, -1, COUNT_BARS)
    assert int(counts[:, 0].sum()) == 2 * nkv * sum(-(-n // tile) for n in lens)
    assert np.array_equal(counts[:, 0], counts[:, 1])
