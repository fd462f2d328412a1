"""Sizes next to what int32 holds (GPU)."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_bounds_of_almost_2_31_frames(pa):
    """1386 heads of 1,549,411 frames are 2^31 - 2 units of work: the table repeats three frames."""
    H, blocks, B, D = 1386, 1549411, 8, 64
    gen = torch.Generator().manual_seed(1)
    kc = torch.randn(3, B, H, D, generator=gen).half().cuda()
    t = (torch.arange(blocks, device="cuda") % 3).to(torch.int32)[None]
    n = torch.tensor([blocks * B], dtype=torch.int32, device="cuda")
    bounds = torch.zeros(3, H, 2, D, dtype=torch.float16, device="cuda")
    pa.pa_block_bounds(kc, t, n, None, bounds)
    assert pa.pa_get_device_status() == 0
    assert torch.equal(bounds[:, :, 0], kc.amin(1)) and torch.equal(bounds[:, :, 1], kc.amax(1))


def test_selection_of_as_many_places_as_int32_holds(pa):
    K = 2 ** 31 - 1
    t = torch.arange(5, dtype=torch.int32, device="cuda")[None]
    n = torch.tensor([33], dtype=torch.int32, device="cuda")
    bounds = torch.zeros(5, 1, 2, 64, dtype=torch.float16, device="cuda")
    q = torch.ones(1, 1, 64, dtype=torch.float16, device="cuda")
    whole = torch.full((K + 9,), 7, dtype=torch.int32, device="cuda")
    sel = whole[:K].view(1, 1, K)
    pa.pa_select_blocks(q, bounds, t, n, 8, sel)
    assert pa.pa_get_device_status() == 0
    assert sel[0, 0, :5].tolist() == [0, 1, 2, 3, 4]
    for i in range(5, K, 1 << 28):                     # in parts: a comparison makes a byte an entry
        assert bool((sel[0, 0, i:i + (1 << 28)] == -1).all())
    assert (whole[K:] == 7).all()
