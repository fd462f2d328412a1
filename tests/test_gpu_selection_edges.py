"""Edges of pa_select_blocks (GPU): lists that take every frame, and frames that are kept, with bad ids among them."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,bad", [(20, 3), (10, 9), (4, 0), (4, 9), (4, 5)])
@pytest.mark.parametrize("value", [-7, 12])
def test_bad_frame_ids_set_the_status(pa, K, bad, value):
    """10 frames of 12: more places than frames, as many, and fewer, the bad id kept or not."""
    gen = torch.Generator().manual_seed(K)
    S, H, g, D, B = 3, 2, 2, 64, 8
    t = torch.stack([torch.randperm(12, generator=gen)[:10] for _ in range(S)]).int()
    t[1, bad] = value
    lens = torch.tensor([80, 77, 80], dtype=torch.int32).cuda()
    bounds = torch.randn(12, H, 2, D, generator=gen).half().sort(dim=2).values.contiguous().cuda()
    q = torch.randn(S, H * g, D, generator=gen).half().cuda()
    kc, vc = (torch.randn(12, B, H, D, generator=gen).half().cuda() for _ in range(2))
    sel = torch.full((S, H, K), -9, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(q, bounds, t.cuda(), lens, B, sel, keep_first=1, keep_last=1)
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_BLOCK
    listed = bad in (0, 9) or K >= 10
    assert all((bad in sel[1, h].tolist()) == listed for h in range(H))
    assert (sel.sort().values[:, :, -min(K, 10):] >= 0).all() and (sel == -1).sum() == S * H * max(0, K - 10)
    out = torch.full_like(q, float("nan"))
    pa.pa_decode_selected(q, kc, vc, t.cuda(), lens, sel, 0.1, out)
    assert pa.pa_get_device_status() == (pa.PA_DEV_BAD_BLOCK if listed else 0)
    assert bool(out[1].any()) != listed and out[0].any() and out[2].any()
