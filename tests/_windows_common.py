"""Helpers for the tests of the window attention and the 8-bit cache."""

from __future__ import annotations

import numpy as np
import torch

from oracle.windows import Cache8
from tests._operators_common import TD


def attended(lens, fresh, B, window, sinks):
    """For each sequence the table positions of frames that hold a token that one of its last `fresh` queries attends."""
    out = []
    for n, c in zip(lens, fresh):
        start = max(0, n - c + 1 - window) if window else 0
        hold = set(range(-(-min(sinks, n) // B))) | set(range(start // B, -(-n // B)))
        out.append(sorted(hold) if n else [])
    return out


def window_tables(gen, lens, fresh, B, window, sinks, spare=3, gone=-1):
    """(block_tables int32 [S, max_blocks], frames): shuffled frames where a query attends a token, `gone` elsewhere."""
    held = attended(lens, fresh, B, window, sinks)
    nb = sum(map(len, held)) + spare
    order = torch.randperm(nb, generator=gen).tolist()
    tables = torch.full((len(lens), max([-(-n // B) for n in lens] + [1])), gone, dtype=torch.int32)
    for s, frames in enumerate(held):
        for j in frames:
            tables[s, j] = order.pop()
    return tables, nb


def hidden_slots(lens, fresh, B, window, sinks, tables, nb):
    """[nb, B] true where a slot holds no token that a query attends."""
    hide = torch.ones(nb, B, dtype=torch.bool)
    for s, (n, c) in enumerate(zip(lens, fresh)):
        j = torch.arange(n)
        start = max(0, n - c + 1 - window) if window else 0
        j = j[(j >= start) | (j < sinks)]
        hide[tables[s, j // B].long(), j % B] = False
    return hide


def cache8(gen, tables, lens, nb, H, B, D, dtype, spread=1.0):
    """An 8-bit cache of random rows, filled by appends of several lengths, and noise everywhere else."""
    shape = (nb, H, B, D)
    c = Cache8(torch.randint(0, 256, shape, generator=gen).to(torch.uint8).numpy(),
               torch.randn(nb, H, generator=gen).numpy().astype(np.float32))
    for s, n in enumerate(lens):
        at = 0
        while at < n:
            j = at // B
            m = min(n - at, int(torch.randint(1, B + 1, (1,), generator=gen)))
            m = min(m, (j + 1) * B - at)
            if tables[s, j] >= 0:
                scale = torch.exp(spread * torch.randn(1, H, 1, generator=gen))
                c.append(tables[s].numpy(), at + m, (torch.randn(m, H, D, generator=gen) * scale).to(TD[dtype]).float().numpy())
            at += m
    return c


def on_gpu(c: Cache8):
    return torch.from_numpy(c.codes).cuda(), torch.from_numpy(c.steps).cuda()
