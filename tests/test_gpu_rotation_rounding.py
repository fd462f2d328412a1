"""The rotation bit for bit: each product and each sum rounded to fp32 by itself, then once to the cache's type, or coded in
4 bits as the formula says (GPU).  Enough rows that a fused product shows: it moves two fp32 results in five."""

import numpy as np
import pytest
import torch

from oracle.operators import cos_sin_table, quantise_q4, rotate
from tests._operators_common import TD

pytestmark = pytest.mark.gpu


def inputs(dtype, D, R, T, H, Hq, seed):
    g = torch.Generator().manual_seed(seed)
    k, v, q = (torch.randn(T, n, D, generator=g).to(TD[dtype]) for n in (H, H, Hq))
    pos = torch.randint(0, 2000, (T,), generator=g).int()
    return k, v, q, pos, torch.randperm(T, generator=g).int(), cos_sin_table(2000, R)


def turned(x, table, pos, interleaved):
    return rotate(x.float().numpy(), table, pos.numpy(), interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,D,R", [("f32", 128, 128), ("f32", 64, 32), ("f16", 128, 128), ("bf16", 128, 64), ("f16", 80, 48), ("bf16", 64, 64)])
def test_rows(pa, dtype, D, R, interleaved):
    T, H, Hq, B = 2048, 4, 8, 16
    k, v, q, pos, slots, table = inputs(dtype, D, R, T, H, Hq, D + R)
    kc, vc = (torch.zeros(T // B, B, H, D, dtype=TD[dtype], device="cuda") for _ in range(2))
    qo = torch.empty_like(q, device="cuda")
    pa.pa_cache_append_rope(k.cuda(), v.cuda(), slots.cuda(), kc, vc, pos.cuda(), torch.from_numpy(table).cuda(), q=q.cuda(), q_out=qo,
                            interleaved=interleaved)
    assert pa.pa_get_device_status() == 0
    for got, x in ((kc.flatten(0, 1)[slots.long().cuda()], k), (qo, q)):
        assert torch.equal(got.cpu(), torch.from_numpy(turned(x, table, pos, interleaved)).to(TD[dtype]))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,D,R", [("f16", 128, 128), ("bf16", 128, 96), ("f16", 64, 64), ("bf16", 64, 32)])
def test_codes(pa, dtype, D, R, interleaved):
    T, H, B = 8192, 16, 16
    k, v, q, pos, slots, table = inputs(dtype, D, R, T, H, 1, D + R + 1)
    kc, vc = (torch.zeros(T // B, H, B, 5 * D // 8, dtype=torch.uint8, device="cuda") for _ in range(2))
    pa.pa_cache_append_q4(k.cuda(), v.cuda(), slots.cuda(), kc, vc, pos.cuda(), torch.from_numpy(table).cuda(), interleaved=interleaved)
    assert pa.pa_get_device_status() == 0
    for cache, x in ((kc, turned(k, table, pos, interleaved)), (vc, v.float().numpy())):
        got = cache.transpose(1, 2).flatten(0, 1)[slots.long().cuda()].cpu().numpy()
        assert np.array_equal(got, quantise_q4(x))
