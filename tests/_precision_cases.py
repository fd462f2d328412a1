"""Decode inputs whose scores are exact in fp32, so that what a test sees is one other rounding, and how far an
output over them may be from the 64-bit one."""

from __future__ import annotations

import numpy as np
import torch

from oracle.operators import GROUP, attend, quantise_q4, values_q4
from tests._operators_common import TD, half_step, tiny


def pack_q4(code, step, offset):
    """4-bit rows from codes [..., D] and steps and offsets [..., D / 32]."""
    code = np.asarray(code, np.uint8)
    par = np.stack([step, offset], axis=-1).astype(np.float16)
    return np.concatenate([code[..., 0::2] | (code[..., 1::2] << 4),
                           np.ascontiguousarray(par).view(np.uint8).reshape(*code.shape[:-1], code.shape[-1] // 8)], axis=-1)


def fine_tolerance(q, k, v, scale, dtype, weight_step, weight_tiny=0.0):
    """[Hq, D]: how far attention of q [Hq, D] over k, v [N, H, D] may be from 64 bits where every score is exact in
    fp32.  In units of the largest weight:

    * a score: its product with scale * log2(e), that factor itself (three roundings) and the difference from the
      running maximum are off by 6 * 2^-24 of the largest score at most, and a weight by that share;
    * a weight: 2^-22 for each of up to three exponentials (its own, a rescaling, a join), weight_step for its
      rounding to the tensor cores' type and weight_tiny where that type has no smaller numbers;
    * sums of N terms in fp32, each off by at most 2^-23 of a partial sum.
    Weighted values are off by that share of sum w |v|, the sum of weights by the same share; then the output's own
    rounding.
    """
    N, H, _ = k.shape
    g = q.shape[0] // H
    tol = np.empty(q.shape)
    ref = attend(q, k, v, scale)
    for j in range(q.shape[0]):
        a = k[:, j // g] @ q[j] * scale
        w = np.exp(a - a.max())
        mean = w @ np.abs(v[:, j // g]) / w.sum()
        e = 6 * 2.0 ** -24 * np.abs(a).max() + 3 * 2.0 ** -22 + weight_step + N * 2.0 ** -23
        tol[j] = e * (mean + np.abs(ref[j])) + weight_tiny * np.abs(v[:, j // g]).sum(0) / w.sum()
    return tol + half_step(TD[dtype]) * np.abs(ref) + tiny(TD[dtype])


def single_products(H, g, D, N, seed):
    """Queries of one element each and keys whose groups lie far from zero: a score is one product of up to about +-60,
    all within a few of one another, and a key's rounding to fp16 moves it by up to 0.015.  -> q [H g, D] (bf16
    numbers), 4-bit keys and values [N, H, W]."""
    rng = np.random.default_rng(seed)
    centre = np.repeat(rng.choice([-1, 1], D // GROUP) * rng.uniform(8, 12, D // GROUP), GROUP)
    k = quantise_q4((0.3 * rng.standard_normal((N, H, D)) + centre).astype(np.float32))
    v = quantise_q4(rng.standard_normal((N, H, D)).astype(np.float32))
    top = np.abs(values_q4(k)).max((0, 1))
    q = np.zeros((H * g, D))
    for j in range(H * g):
        d = int(rng.integers(D))
        q[j, d] = float(torch.tensor(60.0 / top[d]).bfloat16())
    return q, k, v


def outlying_query(H, g, D, N, seed):
    """One query element 2^21 times the others, where all keys are 0, and groups of 32 keys that are one number each, a
    token's own: a score is 32 times the sum of these, and the whole of it the offsets'."""
    rng = np.random.default_rng(seed)
    offset = rng.integers(-512, 513, (N, H, D // GROUP)) / 256.0
    offset[..., 0] = 0
    k = pack_q4(np.zeros((N, H, D)), np.zeros_like(offset), offset)
    v = quantise_q4(rng.standard_normal((N, H, D)).astype(np.float32))
    q = np.full((H * g, D), 2.0 ** -4)
    q[:, 5] = 2.0 ** 17
    return q, k, v


def uneven_weights(H, D, part, seed):
    """64 keys whose weights all round the same way to type `part`, seen from the sign of their values: what that
    rounding leaves over adds up, while the weighted values cancel.  A score is the sum of elements 0 and 32 of its key,
    a multiple of 2^-10.  -> keys and values [64, H, D], exact in bf16 and in constant groups of 32."""
    rng = np.random.default_rng(seed)
    j = np.arange(1, 1024)
    w = np.exp(-j / 1024.0)
    left = (w - torch.from_numpy(w).to(part).double().numpy()) / w
    eps = torch.finfo(part).eps
    up, down = j[left > 0.2 * eps], j[left < -0.2 * eps]
    pairs = []
    for a in rng.permutation(up):
        b = down[np.abs(down - a).argmin()]
        if abs(int(b) - int(a)) <= 40 and all(abs(b - p[1]) > 0 for p in pairs):
            pairs.append((int(a), int(b)))
        if len(pairs) == 31:
            break
    assert len(pairs) == 31
    at, sign = [0, 0], [0.0, 0.0]                     # the largest score, twice
    for a, b in pairs:
        at += [a, b]
        sign += [1.0, -1.0]
    at, sign = np.array(at), np.array(sign)
    order = np.concatenate([[0], 1 + rng.permutation(63)])
    k, v = np.zeros((64, H, D)), np.zeros((64, H, D))
    k[:, :, :32] = -(at[order] // 32 / 32.0)[:, None, None]
    k[:, :, 32:64] = -(at[order] % 32 / 1024.0)[:, None, None]
    v[:] = sign[order][:, None, None]
    return k, v


def one_sink(H, D, N):
    """One key far above all others, its value zero: the output is what the others' small weights leave, each
    0.69 * 2^-24 of the sink's.  -> keys and values [N, H, D] in constant groups of 32."""
    k, v = np.full((N, H, D), -17.0), np.ones((N, H, D))
    k[N // 2], v[N // 2] = 0.0, 0.0
    k[:, :, 32:] = 0.0
    return k, v


def paged_rows(rows, B, seed):
    """Rows [N, H, W] of one sequence in shuffled frames of B: (cache as [frames, B, H, W], table [1, frames])."""
    n = -(-len(rows) // B)
    order = torch.randperm(n + 2, generator=torch.Generator().manual_seed(seed))[:n]
    cache = torch.zeros(n + 2, B, *rows.shape[1:], dtype=rows.dtype)
    for j in range(n):
        part = rows[j * B:(j + 1) * B]
        cache[order[j], : len(part)] = part
    return cache, order.to(torch.int32)[None]
