"""A serving step around the attention -- oracle (test infrastructure).

Norms and rotations of heads in float64, the angles from exact integers; page
plans and trims as loops over sequences and tokens.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

# pi to 60 digits, as a fraction.
PI = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)


def cos_sin(positions, inv_freq):
    """cos and sin [rows, len(inv_freq)] of positions[r] * inv_freq[i], the float64
    inv_freq taken as exact and the angle reduced to half a turn in 128 bits."""
    turns = [round(Fraction(float(f)) / (2 * PI) * 2 ** 128) for f in inv_freq]
    part = [[(int(p) * f + 2 ** 127) % 2 ** 128 - 2 ** 127 for f in turns] for p in positions]
    angle = 2 * np.pi * np.array(part, dtype=object).astype(np.float64).reshape(len(positions), len(turns)) / 2.0 ** 128
    return np.cos(angle), np.sin(angle)


def norm_rope_ref(x, positions, inv_freq, weight=None, eps=1e-6, interleaved=False, scale=1.0):
    """float64 heads [rows, heads, HD], normed and rotated; and, for error bounds,
    |y_a| + |y_b| of each value's pair (|y| where it does not turn)."""
    y = np.asarray(x, dtype=np.float64).copy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    rot = 2 * len(inv_freq)
    out, size = y.copy(), np.abs(y)
    if rot:
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        cos, sin = (scale * t[:, None] for t in cos_sin(positions, inv_freq))
        out[..., a] = y[..., a] * cos - y[..., b] * sin
        out[..., b] = y[..., b] * cos + y[..., a] * sin
        size[..., a] = size[..., b] = abs(scale) * (np.abs(y[..., a]) + np.abs(y[..., b]))
    return out, size


def plan_ref(have, new, free, table, page, num_rows):
    """One step's plan.  free: list of pages, the last goes first; table: int array,
    changed in place, as free is.  Returns (lens, row_starts, positions, slots, fine)."""
    cols, wanted, at, fine = table.shape[1], 0, 0, True
    lens, starts = list(have), [0]
    positions, slots = np.full(num_rows, -1), np.full(num_rows, -1)
    held = len(free)
    for b, (h, n) in enumerate(zip(have, new)):
        n = max(n, 0) if h >= 0 else 0
        old, total = -(-h // page), -(-(h + n) // page)
        room = total <= cols
        if h >= 0 and room:
            wanted += total - old
        served = h >= 0 and room and (total == old or wanted <= held) and (n == 0 or at + n <= num_rows)
        if served:
            for c in range(old, total):
                table[b, c] = free.pop()
            for i in range(n):
                positions[at + i] = h + i
                slots[at + i] = table[b, (h + i) // page] * page + (h + i) % page
            lens[b] = h + n
        fine = fine and (served or h < 0)
        at += n
        starts.append(at)
    return lens, starts, positions, slots, fine


def trim_ref(lens, keep, free, table, page):
    """Pages behind the kept tokens go back to the list, in place: the last of them first."""
    back = []
    for b, (n, k) in enumerate(zip(lens, keep)):
        if 0 <= k < n:
            back += [int(table[b, c]) for c in range(-(-k // page), -(-n // page))]
    free.extend(reversed(back))
