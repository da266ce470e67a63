"""Paged caches for the GPU tests: pools between canary bands, scattered block
tables, and the oracle's view of them."""
from __future__ import annotations

import numpy as np
import torch

import long_context_chunked_gb300 as cp
import oracle

BAND = 4096  # canary bytes on each side of a buffer
CANARY = 0x7E


class Buffer:
    """A device tensor between canary bands."""

    def __init__(self, array: np.ndarray, dtype: torch.dtype):
        self.array = np.ascontiguousarray(array)
        raw = torch.from_numpy(self.array.reshape(-1).view(np.uint8).copy())
        self.n = raw.numel()
        self.base = torch.full((BAND + self.n + BAND,), CANARY, dtype=torch.uint8, device="cuda")
        self.base[BAND:BAND + self.n] = raw.cuda()
        self.t = self.base[BAND:BAND + self.n].view(dtype).view(self.array.shape)

    def host(self) -> np.ndarray:
        return self.base[BAND:BAND + self.n].cpu().numpy().view(self.array.dtype).reshape(
            self.array.shape)

    def intact(self) -> bool:
        return bool((self.base[:BAND] == CANARY).all() and (self.base[BAND + self.n:] == CANARY).all())


def bf16_normal(rng, *shape) -> np.ndarray:
    return oracle.bf16_bits(torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(
        torch.bfloat16))


def i32(values) -> torch.Tensor:
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


class Paged:
    """A paged cache whose slots all hold NaN until something is written, and
    whose table names pages in random order.  Columns behind a sequence's
    capacity name pages that do not exist: they must never be read."""

    def __init__(self, nkv, hd, page, caps, e4m3, seed=0, spare_pages=3, stride_pad=2):
        rng = np.random.default_rng(seed)
        need = [-(-c // page) for c in caps]
        n = sum(need) + spare_pages
        self.page, self.e4m3, self.nkv, self.hd = page, e4m3, nkv, hd
        cols = max(max(need), 1)
        order = rng.permutation(n)
        self.table = np.full((len(caps), cols + stride_pad), 2 ** 30, np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        shape = (n, nkv, page, hd)
        if e4m3:
            self.pools = [np.full(shape, 0x7F, np.uint8) for _ in range(2)]
            self.scales = [np.full(shape[:3], np.nan, np.float32) for _ in range(2)]
            dt = torch.float8_e4m3fn
        else:
            self.pools = [np.full(shape, 0x7FC1, np.uint16) for _ in range(2)]
            self.scales, dt = None, torch.bfloat16
        self.dt = dt
        self.cols = cols

    def upload(self):
        self.d_pools = [Buffer(x, self.dt) for x in self.pools]
        self.d_scales = None if self.scales is None else [Buffer(x, torch.float32) for x in self.scales]
        self.d_table = Buffer(self.table, torch.int32)
        ks, vs = (None, None) if self.d_scales is None else (s.t for s in self.d_scales)
        self.kv = cp.PagedKV(self.d_pools[0].t, self.d_pools[1].t, self.d_table.t[:, :self.cols], ks, vs)
        return self

    def fill(self, rng, lens):
        """The oracle writes lens[b] tokens of N(0,1) into every sequence."""
        starts = np.concatenate([[0], np.cumsum(np.maximum(lens, 0))])
        new = [bf16_normal(rng, starts[-1], self.nkv, self.hd) for _ in range(2)]
        oracle.paged_write_ref(self.pools, self.scales, self.table, self.page, [0] * len(lens),
                               starts, new)

    def check_pools(self):
        """The device pools hold the oracle's, bit for bit (NaN scales alike)."""
        for d, h in zip(self.d_pools, self.pools):
            assert np.array_equal(d.host(), h)
        for d, h in zip(self.d_scales or [], self.scales or []):
            assert np.array_equal(d.host(), h, equal_nan=True)

    def intact(self) -> bool:
        bufs = self.d_pools + (self.d_scales or []) + [self.d_table]
        return all(b.intact() for b in bufs) and np.array_equal(self.d_table.host(), self.table)


# Error bound of a bf16 attention output against float64 (one softmax row):
#   the output's rounding        2^-8 |O|                      (half a bf16 step)
#   a probability's rounding     2^-11 A, A = sum p |v| / l    (fp16; a bf16 pair is finer)
#   the logits' fp32 products    HD * 2^-23 X in the exponent, X = max_t scale sum |q k|,
#                                so a factor e^(that) on every p: A times twice it
#   exponentials, l, O sums      2^-20 A                       (fp32)
def out_bound(ref, A, X, hd):
    dx = hd * 2.0 ** -23 * X[..., None]
    return 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -10) + A * (2.0 ** -11 + 2 * dx + 2.0 ** -20) + 1e-37


def lse_bound(lse, X, hd):
    """The logits' error, and the fp32 rounding of m + log2 l and its factor."""
    return hd * 2.0 ** -23 * X + 2.0 ** -21 * (np.abs(np.where(np.isfinite(lse), lse, 0)) + 1)


def check_decode(out, lse, ref, ref_lse, A, X, hd):
    err = np.abs(out - ref)
    bound = out_bound(ref, A, X, hd)
    assert np.all(err <= bound), f"worst {np.max(err / bound):.3f} of the bound"
    if lse is not None:
        empty = np.isinf(ref_lse)
        assert np.array_equal(np.isneginf(lse), empty)
        d = np.abs(lse[~empty] - ref_lse[~empty])
        assert np.all(d <= lse_bound(ref_lse, X, hd)[~empty]), f"lse off by {d.max():.3e}"
