"""The paged KV cache -- oracle (test infrastructure).

Pages [num_pages, NKV, page_size, HD]; token t of sequence b sits in page
table[b][t div page_size] at slot t mod page_size.  e4m3 pages store
    s = max(amax, 2^-110) / 448,   x8 = e4m3(x * (448 / max(amax, 2^-110)))
with every operation rounded to float32 and the last one to the nearest e4m3
value (ties to the even mantissa); the value read back is s * x8.  e2m1 pages
hold two 4-bit codes to a byte, the first in the lower half, and for each row a
record of 4 + HD/32 bytes, s as float32 and an e4m3 code r_g for each group of
32 values:
    s = 2^(floor(log2(max(amax, 2^-117))) - 9),   r_g = e4m3(amax_g / (6 s)),
    x4 = e2m1((x / s) / r_g), 0 where r_g = 0;
the value read back is s * r_g * x4.  The attention is float64 over those values.
"""
from __future__ import annotations

import numpy as np

from .striped import bits_to_f64

TINY_AMAX = np.float32(2.0 ** -110)
TINY_AMAX4 = 2.0 ** -117
GROUP4 = 32
E2M1_MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


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


def to_e2m1(x: np.ndarray) -> np.ndarray:
    """Codes of the nearest e2m1 values (ties to the even code, 6 at most; -0 is
    taken as 0), by search."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 6.0)
    hi = np.clip(np.searchsorted(E2M1_MAGNITUDES, a), 1, 7)
    lo = hi - 1
    dl, dh = a - E2M1_MAGNITUDES[lo], E2M1_MAGNITUDES[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(x < 0, code | 8, code).astype(np.uint8)


def quantise4_rows(x: np.ndarray):
    """float64 rows [..., HD] -> (bytes [..., HD/2], records [..., 4 + HD/32])."""
    x = np.asarray(x, dtype=np.float64)
    fine = np.isfinite(x).all(-1)
    x = np.where(fine[..., None], x, 0.0)
    groups = x.reshape(*x.shape[:-1], -1, GROUP4)
    amax_g = np.abs(groups).max(-1)
    s = np.ldexp(1.0, np.frexp(np.maximum(amax_g.max(-1), TINY_AMAX4))[1] - 10)
    r = to_e4m3(amax_g / s[..., None] / 6)
    unit = s[..., None] * e4m3_values()[r]
    y = groups / np.where(unit > 0, unit, 1.0)[..., None]
    code = np.where((unit > 0)[..., None], to_e2m1(y), 0).reshape(x.shape)
    code[~fine], r[~fine] = 0, 0
    s32 = np.where(fine, s, np.nan).astype(np.float32)
    rec = np.concatenate([np.ascontiguousarray(s32[..., None]).view(np.uint8), r], -1)
    return (code[..., ::2] | (code[..., 1::2] << 4)).astype(np.uint8), rec


def values4(codes: np.ndarray, rec: np.ndarray) -> np.ndarray:
    """float64 rows of e2m1 bytes and their records (exact)."""
    x = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    mag = E2M1_MAGNITUDES[x & 7]
    s = np.ascontiguousarray(rec[..., :4]).view(np.float32).astype(np.float64)
    unit = s * e4m3_values()[rec[..., 4:]]
    return np.where(x >> 3, -mag, mag) * np.repeat(unit, GROUP4, -1)


def paged_write_ref(pools, scales, table, page_size, cache_lens, row_starts, new):
    """Write rows of `new` (pair of bf16 bit arrays [rows, NKV, HD]) into the
    pools (pair; bf16 bits, or e4m3 codes when scales is a pair, or e2m1 bytes
    when it is one of records) in place."""
    for b, have in enumerate(cache_lens):
        if have < 0:
            continue
        for row in range(row_starts[b], row_starts[b + 1]):
            t = have + row - row_starts[b]
            page, slot = table[b][t // page_size], t % page_size
            for i in range(2):
                if scales is None:
                    pools[i][page, :, slot] = new[i][row]
                elif scales[i].ndim == 4:
                    pools[i][page, :, slot], scales[i][page, :, slot] = quantise4_rows(
                        bits_to_f64(new[i][row]))
                else:
                    pools[i][page, :, slot], scales[i][page, :, slot] = quantise_rows(new[i][row])


def paged_rows(pool, scale, table_row, page_size, first, n):
    """float64 values [n - first, NKV, HD] of tokens first .. n-1 of one sequence."""
    t = np.arange(first, n)
    page, slot = np.asarray(table_row)[t // page_size], t % page_size
    x = pool[page, :, slot]
    if scale is None:
        return bits_to_f64(x)
    if scale.ndim == 4:
        return values4(x, scale[page, :, slot])
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
