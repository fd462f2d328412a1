"""Inputs of the window decode and of the decode over the 8-bit cache whose scores are exact in fp32 but for the products that
each test names, and how far an output over them may be from the 64-bit one."""

from __future__ import annotations

import numpy as np
import torch

from oracle.operators import attend
from tests._operators_common import TD
from tests._precision_cases import fine_tolerance


class Rows8:
    """One sequence's rows of the 8-bit cache: whole numbers of -127 .. 127 [N, H, D] and, for each row, its frame's step [N, H]."""

    def __init__(self, codes, steps, B=16):
        self.codes = np.asarray(codes, np.int64)
        self.steps = np.asarray(steps, np.float32)
        assert np.abs(self.codes).max() <= 127 and self.steps.shape == self.codes.shape[:2]
        for j in range(0, len(self.steps), B):
            assert (self.steps[j:j + B] == self.steps[j]).all()

    def values(self):
        return self.codes * self.steps.astype(np.float64)[..., None]


def tolerance8(q, k, v, scale, dtype):
    """[Hq, D] for rows k, v of the 8-bit cache: as fine_tolerance, with one rounding more of a score (its product with the step) and
    of a weight (the same), a weight carried to 2^-22 of itself, and where the two fp16 parts have no smaller numbers to half of
    fp16's least, 2^-25, of a weight that is held 2^7 higher at least and a step of 1/2 at least where it is the largest:
    2^-31 of the largest weight times the largest step, for each key."""
    kk, vv = k.values(), v.values()
    tol = fine_tolerance(q, kk, vv, scale, dtype, 2.0 ** -22 + 2.0 ** -24)
    g = q.shape[0] // kk.shape[1]
    for j in range(len(q)):
        h = j // g
        a = kk[:, h] @ q[j] * scale
        w = np.exp(a - a.max())
        more = 2.0 ** -24 * np.abs(a).max()
        tol[j] += more * 2 * (w @ np.abs(vv[:, h])) / w.sum()
        tol[j] += 2.0 ** -31 * float(v.steps[:, h].max()) * np.abs(v.codes[:, h]).sum(0) / w.sum()
    return tol


def spread_sum(total, dims):
    """`dims` whole numbers of 0 .. 127 whose sum is `total`, as equal as they can be."""
    out = np.full(dims, total // dims)
    out[:total % dims] += 1
    assert out.max() <= 127
    return out


def uneven_weights8(H, D, step, seed):
    """64 keys whose weights, times the step of their values, all round the same way to fp16, seen from the sign of their
    values: what that rounding leaves over adds up while the weighted values cancel.  A score is the sum of the first 16
    elements of its key, a multiple of 2^-10.  -> (q of one head [D], keys, values)."""
    rng = np.random.default_rng(seed)
    j = np.arange(1, 1024)
    w = np.exp(-j / 1024.0) * float(np.float32(step))
    left = (w - w.astype(np.float16).astype(np.float64)) / w
    eps = torch.finfo(torch.float16).eps
    up, down = j[left > 0.2 * eps], j[left < -0.2 * eps]
    pairs = []
    for a in rng.permutation(up):
        b = down[np.abs(down - a).argmin()]
        if abs(int(b) - int(a)) <= 40 and all(b != p[1] for p in pairs):
            pairs.append((int(a), int(b)))
        if len(pairs) == 31:
            break
    assert len(pairs) == 31
    at = np.array([0, 0] + [x for p in pairs for x in p])
    sign = np.array([0, 0] + [1, -1] * 31)
    order = np.concatenate([[0], 1 + rng.permutation(63)])
    k, v = np.zeros((64, H, D), np.int64), np.zeros((64, H, D), np.int64)
    for n, i in enumerate(order):
        k[n, :, :16] = -spread_sum(int(at[i]), 16)
        v[n] = sign[i]
    q = np.zeros(D)
    q[:16] = 1.0
    return q, Rows8(k, np.full((64, H), 2.0 ** -10)), Rows8(v, np.full((64, H), step))


def sink_and_steps(H, D, N, step, others):
    """One key far above all others whose value is zero and whose frame has values in steps of `step`, the largest; the
    others' weights are 0.69 * 2^-24 of its, their values one step of `others` each."""
    k, v = np.zeros((N, H, D), np.int64), np.ones((N, H, D), np.int64)
    k[:, :, 0] = -17
    at = N // 2 // 16 * 16
    k[at], v[at] = 0, 0
    steps = np.full((N, H), others, np.float32)
    steps[at:at + 16] = step
    q = np.zeros(D)
    q[0] = 1.0
    return q, Rows8(k, np.ones((N, H))), Rows8(v, steps)


def parts16(w, parts=2):
    """What numbers are as `parts` fp16 numbers, one the rounding of what the one before left."""
    out = np.zeros_like(w)
    for _ in range(parts):
        out = out + (w - out).astype(np.float16).astype(np.float64)
    return out


def carried(k, v, q, parts=2, room=7, in_units=True):
    """One head's attention with weights carried as the kernel does: times their step in units of the power of two above the
    largest step, 2^room times what they stand for, in `parts` fp16 numbers; everything else in 64 bits.  Mistakes are
    planted by other arguments."""
    a = k.values()[:, 0] @ q
    w = np.exp(a - a.max())
    step = v.steps[:, 0].astype(np.float64)
    unit = 2.0 ** (np.floor(np.log2(step.max())) + 1) if in_units else 1.0
    p = parts16(w * 2.0 ** room * step / unit, parts) * unit / 2.0 ** room
    return p @ v.codes[:, 0] / w.sum()


def hidden_between(rows, sinks, gap, fill):
    """Rows [N, ...] with `gap` others behind the first `sinks`, which a window of N - sinks does not see."""
    rows = np.asarray(rows)
    return np.concatenate([rows[:sinks], np.full((gap, *rows.shape[1:]), fill, rows.dtype), rows[sinks:]])


def rounded(x, dtype):
    return torch.from_numpy(np.asarray(x)).to(TD[dtype]).double().numpy()


def within(got, q, k, v, dtype):
    ref = attend(q, k.values(), v.values(), 1.0)
    return np.abs(got - ref) <= tolerance8(q, k, v, 1.0, dtype)
