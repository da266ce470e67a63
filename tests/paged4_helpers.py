"""4-bit paged caches for the GPU tests, as tests/paged_helpers.py has the others,
and the error bound of attention over them."""
from __future__ import annotations

import numpy as np
import torch

import long_context_chunked_gb300 as cp
import oracle
from paged_helpers import Buffer, Paged, bf16_normal, lse_bound


class Paged4(Paged):
    """An e2m1 cache.  Slots that nothing was written to hold ones in every bit: NaN
    for s, and r_g and codes that no writer makes."""

    def __init__(self, nkv, hd, page, caps, seed=0, spare_pages=3, stride_pad=2):
        super().__init__(nkv, hd, page, caps, False, seed, spare_pages, stride_pad)
        n = self.pools[0].shape[0]
        self.pools = [np.full((n, nkv, page, hd // 2), 0xFF, np.uint8) for _ in range(2)]
        self.scales = [np.full((n, nkv, page, 4 + hd // 32), 0xFF, np.uint8) for _ in range(2)]
        self.dt = torch.uint8

    def fill(self, rng, lens):
        """As Paged.fill, all rows quantised at once."""
        n = np.maximum(lens, 0)
        seq = np.repeat(np.arange(len(n)), n)
        t = np.concatenate([np.arange(i) for i in n])
        page, slot = self.table[seq, t // self.page], t % self.page
        for pool, scale in zip(self.pools, self.scales):
            for at in range(0, len(t), 8192):
                part = slice(at, at + 8192)
                x = oracle.bits_to_f64(bf16_normal(rng, len(t[part]), self.nkv, self.hd))
                pool[page[part], :, slot[part]], scale[page[part], :, slot[part]] = oracle.quantise4_rows(x)

    def upload(self):
        self.d_pools = [Buffer(x, torch.uint8) for x in self.pools]
        self.d_scales = [Buffer(x, torch.uint8) for x in self.scales]
        self.d_table = Buffer(self.table, torch.int32)
        self.kv = cp.PagedKV(self.d_pools[0].t, self.d_pools[1].t, self.d_table.t[:, :self.cols],
                             self.d_scales[0].t, self.d_scales[1].t)
        return self


def largest_product(q, c, lens, scale):
    """max_t p_t s_t / l of each [B, NQ] (s: the V row's scale)."""
    out = np.zeros(q.shape[:2])
    G = q.shape[1] // c.nkv
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        t = np.arange(n)
        k = oracle.paged_rows(c.pools[0], c.scales[0], c.table[b], c.page, 0, n)
        rec = c.scales[1][c.table[b][t // c.page], :, t % c.page]
        s = np.ascontiguousarray(rec[..., :4]).view(np.float32)[..., 0].astype(np.float64)
        for g in range(c.nkv):
            x = scale * (q[b, g * G:(g + 1) * G] @ k[:, g].T)
            e = np.exp(x - x.max(-1, keepdims=True))
            out[b, g * G:(g + 1) * G] = (e * s[:, g]).max(-1) / e.sum(-1)
    return out


# Error bound of the output, as paged_helpers.out_bound but that P is rounded to
# fp16 twice, alone and times r_g / 256 (2^-11 A each), and may fall below fp16's
# normal range: P is p s 2^7 / W with W at most 2 M, M the largest p s, so half of
# fp16's least step, 2^-25, in P or in P times r_g / 256 <= 1.75, times x4 <= 6 and 2^8
# W / 2^7, is at most 1.75 * 6 * 2^-25 * 4 M each: 2^-18 M for both, for every token.
def out_bound4(ref, A, X, M, n, hd):
    dx = hd * 2.0 ** -23 * X[..., None]
    few = np.asarray(n, dtype=np.float64)[:, None, None] * 2.0 ** -18 * M[..., None]
    return 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -9) + A * (2.0 ** -10 * (1 + 2.0 ** -10) + 2 * dx + 2.0 ** -20) \
        + few + 1e-37


def check_decode4(c, q, lens, scale, out, lse=None):
    """q, out [B, NQ, HD] and lse [B, NQ], float64, against the oracle."""
    ref, ref_lse, A, X = oracle.paged_decode_ref(q, c.pools, c.scales, c.table, c.page, lens, scale)
    bound = out_bound4(ref, A, X, largest_product(q, c, lens, scale), np.maximum(lens, 0), c.hd)
    err = np.abs(out - ref)
    assert np.all(err <= bound), f"worst {np.max(err / bound):.3f} of the bound"
    if lse is not None:
        empty = np.isinf(ref_lse)
        assert np.array_equal(np.isneginf(lse), empty)
        d = np.abs(lse[~empty] - ref_lse[~empty])
        assert np.all(d <= lse_bound(ref_lse, X, c.hd)[~empty]), f"lse off by {d.max():.3e}"
    return ref
