"""The paged KV cache -- oracle (test infrastructure).

Pages [num_pages, NKV, page_size, HD]; token t of sequence b sits in page
table[b][t div page_size] at slot t mod page_size.  e4m3 pages store
    s = max(amax, 2^-110) / 448,   x8 = e4m3(x * (448 / max(amax, 2^-110)))
with every operation rounded to float32 and the last one to the nearest e4m3
value (ties to the even mantissa); the value read back is s * x8.  The
attention is float64 over those values.
"""
from __future__ import annotations

import numpy as np

from .striped import bits_to_f64

TINY_AMAX = np.float32(2.0 ** -110)


def e4m3_values() -> np.ndarray:
    """float64 value of each of the 256 e4m3 codes (1 sign, 4 exponent bits of
    bias 7, 3 mantissa bits, no infinities; 0x7F and 0xFF are NaN)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            mag = np.nan
        out[c] = -mag if c >> 7 else mag
    return out


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """Codes of the nearest e4m3 values (ties to even, saturating at 448; NaN
    to 0x7F), by search over the 127 magnitudes."""
    x = np.asarray(x, dtype=np.float64)
    mags = e4m3_values()[:127]                       # ascending, 0 .. 448
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(mags, a), 1, 126)   # mags[hi-1] <= a <= mags[hi]
    lo = hi - 1
    dl, dh = a - mags[lo], mags[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def quantise_rows(bits: np.ndarray):
    """bf16 bit patterns [..., HD] -> (e4m3 codes [..., HD], float32 scales [...])."""
    x = bits_to_f64(bits).astype(np.float32)
    amax = np.maximum(np.abs(x).max(-1), TINY_AMAX)
    amax = np.where(np.isfinite(x).all(-1), amax, np.float32(np.nan)).astype(np.float32)
    with np.errstate(invalid="ignore"):
        inv = np.float32(448) / amax
        return to_e4m3(x * inv[..., None]), amax / np.float32(448)


def paged_write_ref(pools, scales, table, page_size, cache_lens, row_starts, new):
    """Write rows of `new` (pair of bf16 bit arrays [rows, NKV, HD]) into the
    pools (pair; bf16 bits, or e4m3 codes when scales is a pair) in place."""
    for b, have in enumerate(cache_lens):
        if have < 0:
            continue
        for row in range(row_starts[b], row_starts[b + 1]):
            t = have + row - row_starts[b]
            page, slot = table[b][t // page_size], t % page_size
            for i in range(2):
                if scales is None:
                    pools[i][page, :, slot] = new[i][row]
                else:
                    pools[i][page, :, slot], scales[i][page, :, slot] = quantise_rows(new[i][row])


def paged_rows(pool, scale, table_row, page_size, first, n):
    """float64 values [n - first, NKV, HD] of tokens first .. n-1 of one sequence."""
    t = np.arange(first, n)
    page, slot = np.asarray(table_row)[t // page_size], t % page_size
    x = pool[page, :, slot]
    if scale is None:
        return bits_to_f64(x)
    # s * x8 in float64 is exact; the reader rounds it once
    return e4m3_values()[x] * scale[page, :, slot][..., None].astype(np.float64)


def paged_decode_ref(q, pools, scales, table, page_size, lens, scale):
    """O [B, NQ, HD], LSE [B, NQ] and, for error bounds, A = sum_t p_t |v_t| / l
    [B, NQ, HD] and X = max_t scale * sum_d |q_d k_d| [B, NQ]."""
    B, NQ, HD = q.shape
    NKV = pools[0].shape[1]
    G = NQ // NKV
    out, lse = np.zeros((B, NQ, HD)), np.full((B, NQ), -np.inf)
    A, X = np.zeros((B, NQ, HD)), np.zeros((B, NQ))
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        k, v = (paged_rows(pools[i], None if scales is None else scales[i], table[b], page_size,
                           0, n) for i in range(2))
        for g in range(NKV):
            h = slice(g * G, (g + 1) * G)
            s = scale * (q[b, h] @ k[:, g].T)
            m = s.max(-1, keepdims=True)
            e = np.exp(s - m)
            tot = e.sum(-1, keepdims=True)
            out[b, h] = e @ v[:, g] / tot
            lse[b, h] = (m + np.log(tot))[:, 0]
            A[b, h] = e @ np.abs(v[:, g]) / tot
            X[b, h] = (scale * (np.abs(q[b, h]) @ np.abs(k[:, g]).T)).max(-1)
    return out, lse, A, X
