"""Helpers for the tests of the rotating append, the 4-bit cache and the block-sparse decode."""

from __future__ import annotations

import numpy as np
import torch

TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def host64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def half_step(dtype) -> float:
    """Half a rounding step of a type, relative to the value."""
    return torch.finfo(dtype).eps / 2


def tiny(dtype) -> float:
    """Half the spacing of the type's subnormal numbers: what a rounding near zero is off by."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def paged(gen, lens, B, spare=5, width=None):
    """(block_tables int32 [S, max_blocks] on the GPU, frames): shuffled frames, -1 behind the last."""
    blocks = [-(-n // B) for n in lens]
    nb = sum(blocks) + spare
    order = torch.randperm(nb, generator=gen).tolist()
    width = max(blocks + [1]) if width is None else width
    tables = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(blocks):
        tables[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return tables, nb


def attention_tolerance(ref, dtype, q, k, v, scale, weight_step):
    """How far an attention output may be from the 64-bit one.

    * the output's own rounding: half a step of its type;
    * a score: D products summed in fp32, each sum off by at most a whole step (2^-23) of a partial sum,
      which is at most sum |q_d k_d| <= |q| |k|; the product with scale * log2(e) and the difference from
      the running maximum add two roundings of a number below |q| |k| scale;
    * a weight: 2^-22 from the exponential and its rescalings, weight_step from its rounding, and 2^-24 of the largest weight where it is held in fewer bits
      (a weight below 2^-14 of the reference maximum, of which the running one may be 2^8 short);
    * the sums of weights and of weighted values: fp32, N terms, each sum off by at most 2^-23 of a partial sum.
    A weight that is off by a share e moves the output by at most e * max |v - out| <= 2 e max |v|.
    """
    if not len(k):
        return np.zeros_like(ref)
    D, N = q.shape[-1], len(k)
    reach = np.linalg.norm(q, axis=-1).max() * np.linalg.norm(k, axis=-1).max() * abs(scale)
    e = (D + 4) * 2.0 ** -23 * reach + 2.0 ** -22 + weight_step + 2 * N * 2.0 ** -23
    return half_step(dtype) * np.abs(ref) + 2 * e * np.abs(v).max() + tiny(dtype)
