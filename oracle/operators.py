"""Plain forms of the rotating append, the 4-bit cache and the block-sparse decode.

NumPy only.  Rotation, attention and bounds in 64 bits; what the library defines bit by bit
(4-bit codes, the selection score's sum) in the 32-bit steps of that definition.
"""

from __future__ import annotations

import numpy as np

GROUP = 32
TOP = np.float32(65024.0)  # the top code, 15 rounded steps above -TOP, is at most 65024 (1 + 2^-10): finite in fp16


def cos_sin_table(max_pos: int, rot: int, base: float = 10000.0) -> np.ndarray:
    """[max_pos, rot] float32: cosines, then sines, of position * base^(-2 i / rot)."""
    angle = np.arange(max_pos, dtype=np.float64)[:, None] * base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)


def rotate(x: np.ndarray, table: np.ndarray, positions, interleaved: bool) -> np.ndarray:
    """Rows x [T, H, D] with their first R elements rotated, in x's own precision (float64 or float32,
    each product and sum rounded by itself)."""
    rot = table.shape[1]
    row = table[np.asarray(positions)].astype(x.dtype)
    c, s = row[:, None, : rot // 2], row[:, None, rot // 2:]
    y = x.copy()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def quantise_q4(x: np.ndarray) -> np.ndarray:
    """Rows x [..., D] float32 as 4-bit rows, uint8 [..., 5 D / 8]."""
    x = np.asarray(x, np.float32)
    D = x.shape[-1]
    g = x.reshape(*x.shape[:-1], D // GROUP, GROUP)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], np.float32(0), np.clip(g, -TOP, TOP))
    off = g.min(-1).astype(np.float16)
    step = ((g.max(-1) - off.astype(np.float32)) * (np.float32(1) / np.float32(15))).astype(np.float16)
    st = step.astype(np.float32)[..., None]
    n = np.rint((g - off.astype(np.float32)[..., None]) / np.where(st > 0, st, np.float32(1)))
    n = np.where(st > 0, np.clip(n, 0, 15), 0).astype(np.uint8).reshape(x.shape)
    nan = np.array(0x7FFF, np.uint16).view(np.float16)
    par = np.stack([np.where(bad, nan, step), np.where(bad, nan, off)], axis=-1).astype(np.float16)
    return np.concatenate([n[..., 0::2] | (n[..., 1::2] << 4),
                           np.ascontiguousarray(par).view(np.uint8).reshape(*x.shape[:-1], D // 8)], axis=-1)


def values_q4(rows: np.ndarray, rounded: bool = True) -> np.ndarray:
    """The numbers (float64, each exact in fp16) that 4-bit rows [..., 5 D / 8] stand for; step * n + offset itself
    where not `rounded`."""
    D = rows.shape[-1] // 5 * 8
    code = np.stack([rows[..., : D // 2] & 15, rows[..., : D // 2] >> 4], axis=-1).reshape(*rows.shape[:-1], D // GROUP, GROUP)
    par = np.ascontiguousarray(rows[..., D // 2:]).view(np.float16).reshape(*rows.shape[:-1], D // GROUP, 2).astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        x = code * par[..., :1] + par[..., 1:]
        x = x.astype(np.float16).astype(np.float64) if rounded else x
    return x.reshape(*rows.shape[:-1], D)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float) -> np.ndarray:
    """Attention of queries q [Hq, D] over k, v [N, H, D] in 64 bits, query head j over key head j // (Hq / H);
    zeros where N is 0."""
    N, H, D = k.shape
    if N == 0:
        return np.zeros(q.shape)
    out = np.empty(q.shape)
    g = q.shape[0] // H
    for j in range(q.shape[0]):
        a = k[:, j // g] @ q[j].astype(np.float64) * scale
        w = np.exp(a - a.max())
        out[j] = w @ v[:, j // g] / w.sum()
    return out


def block_bounds(k_frames: np.ndarray, n: int) -> np.ndarray:
    """[H, 2, D] smallest and largest key of the first n tokens of one frame [B, H, D]."""
    return np.stack([k_frames[:n].min(0), k_frames[:n].max(0)], axis=1)


def block_scores(q: np.ndarray, bounds: np.ndarray) -> np.ndarray:
    """Scores [N, H] of N frames' bounds [N, H, 2, D] for queries q [Hq, D], float32: products, then sums of
    neighbours until one is left, then the largest over the queries of a head."""
    N, H, _, D = bounds.shape
    g = q.shape[0] // H
    qq = q.astype(np.float32).reshape(1, H, g, D)
    lo, hi = bounds[:, :, 0, None].astype(np.float32), bounds[:, :, 1, None].astype(np.float32)
    x = qq * np.where(qq >= 0, hi, lo)
    while x.shape[-1] > 1:
        x = x[..., 0::2] + x[..., 1::2]
    return x[..., 0].max(-1)


def select_blocks(scores: np.ndarray, K: int, keep_first: int, keep_last: int) -> np.ndarray:
    """[H, K] int32 from scores [N, H]: the K largest ranks in ascending position, -1 behind the last."""
    N, H = scores.shape
    keep = (np.arange(N) < keep_first) | (np.arange(N) >= N - keep_last)
    out = np.full((H, K), -1, np.int32)
    for h in range(H):
        # every kept frame ranks the same: the lower position first
        rank = np.where(keep, 0.0, -scores[:, h].astype(np.float64))
        order = np.lexsort((np.arange(N), rank, ~keep))[: min(K, N)]
        out[h, : len(order)] = np.sort(order)
    return out
