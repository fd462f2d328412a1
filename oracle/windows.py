"""Plain forms of the window attention and the 8-bit cache.

NumPy only.  Attention in 64 bits; what the library defines bit by bit (8-bit codes and steps) in the 32-bit steps of
that definition.
"""

from __future__ import annotations

import numpy as np

from .operators import attend

LEAST, MOST = np.float32(2.0 ** -60), np.float32(2.0 ** 60)


def seen(p: int, window: int, sinks: int) -> np.ndarray:
    """Positions that a query at position p attends, ascending; every one up to p where window is 0."""
    j = np.arange(p + 1)
    return j if window == 0 else j[(j > p - window) | (j < sinks)]


def attend_seen(q: np.ndarray, k: np.ndarray, v: np.ndarray, p: int, window: int, sinks: int, scale: float) -> np.ndarray:
    """One query [Hq, D] at position p over a sequence's keys and values [N, H, D]; zeros where p is -1."""
    j = seen(p, window, sinks)
    return attend(q, k[j], v[j], scale)


def _top_bits(x: np.float32, nearest: bool) -> np.float32:
    """x > 0 with its 8 leading bits, cut or rounded to even."""
    b = int(np.float32(x).view(np.uint32))
    if nearest:
        b += 0x7FFF + ((b >> 16) & 1)
    return np.uint32(b & 0xFFFF0000).view(np.float32)


def largest_kept(x: np.ndarray, dtype: str) -> np.ndarray:
    """Outputs over the 8-bit cache before they are rounded to `dtype`: codes may stand for up to half a step more than the element they
    came from, so in fp16 a number beyond its largest is that one.  NaN stays."""
    return np.clip(x, -65504.0, 65504.0) if dtype == "f16" else x


class Cache8:
    """An 8-bit cache: codes uint8 [num_blocks, H, B, D], steps float32 [num_blocks, H]."""

    def __init__(self, codes: np.ndarray, steps: np.ndarray):
        self.codes, self.steps = codes, steps

    def append(self, table, length: int, rows: np.ndarray) -> None:
        """rows [n, H, D] as the last n of a sequence's `length` tokens."""
        B = self.codes.shape[2]
        first = length - len(rows)
        rows = np.asarray(rows, np.float32)
        for j in range(first // B, -(-length // B)) if len(rows) else ():
            f = int(table[j])
            lo, hi = max(first, j * B), min(length, (j + 1) * B)
            self._fill(f, lo - j * B, rows[lo - first:hi - first])

    def _fill(self, f: int, at: int, rows: np.ndarray) -> None:
        """rows [n, H, D] at offset `at` of frame f, whose tokens before that stand."""
        for h in range(rows.shape[1]):
            x = rows[:, h]
            old, step = self.codes[f, h, :at], self.steps[f, h]
            sound = np.isfinite(x).all() and (at == 0 or 2.0 ** -67 <= step <= 2.0 ** 60)
            if not sound:
                self.steps[f, h] = np.nan
                self.codes[f, h, at:at + len(x)] = 128
                continue
            x = np.clip(x, -MOST, MOST)
            largest = np.maximum(np.abs(x).max(), LEAST)
            if at == 0:
                r = _top_bits(np.float32(127) / largest, False)
                self.steps[f, h] = np.float32(1) / r
            else:
                r = _top_bits(np.float32(1) / step, True)
                k = 0
                while float(largest) * float(r) > 127 * 2.0 ** k:
                    k += 1
                r = np.float32(r * np.float32(2.0 ** -k))
                self.steps[f, h] = step * np.float32(2.0 ** k)
                if k:
                    old[:] = np.rint((old.astype(np.float64) - 128) / 2.0 ** k) + 128
            self.codes[f, h, at:at + len(x)] = np.rint(x.astype(np.float64) * float(r)) + 128

    def values(self, table, length: int) -> np.ndarray:
        """The numbers that a sequence's tokens stand for, float64 [length, H, D]."""
        B = self.codes.shape[2]
        f, o = np.asarray(table)[np.arange(length) // B].astype(int), np.arange(length) % B
        return (self.codes[f, :, o].astype(np.float64) - 128) * self.steps[f].astype(np.float64)[..., None]
