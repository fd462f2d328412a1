"""Rows next to the end of fp16's range in the 8-bit cache: read back and attended, they stay finite (GPU)."""

import numpy as np
import pytest
import torch

from oracle.windows import Cache8, attend_seen, largest_kept
from tests._operators_common import TD, attention_tolerance, host64, paged
from tests._windows_common import on_gpu

pytestmark = pytest.mark.gpu


def filled(frames, H, B, D, dtype, firsts):
    """Frames of rows +-x, x the frame's number of `frames`, behind a first row +-y, y of `firsts` (None: none); appended on both sides."""
    import paged_kv_cache_126_gb300 as pa

    n = len(frames)
    sign = torch.where(torch.arange(D) % 3 == 0, -1.0, 1.0)
    x = torch.tensor(frames)[:, None, None, None] * sign.expand(n, B, H, D)
    y = torch.tensor([f or 0.0 for f in firsts])[:, None, None] * sign.expand(n, H, D)
    c = Cache8(np.zeros((n, H, B, D), np.uint8), np.zeros((n, H), np.float32))
    codes, steps = on_gpu(c)
    tables = torch.arange(n, dtype=torch.int32)[:, None]
    for upto, rows in ((1, y[:, None]), (B, x)):
        fresh = [(1 if upto == 1 else B - 1) if f is not None else (0 if upto == 1 else B) for f in firsts]
        new = torch.cat([rows[i, :m] for i, m in enumerate(fresh)]).to(TD[dtype])
        if not len(new):
            continue
        lens = torch.tensor([upto if m else 0 for m in fresh], dtype=torch.int32)
        start = torch.tensor(np.cumsum([0] + fresh), dtype=torch.int32)
        pa.pa_cache_append_q8(new.cuda(), new.cuda(), tables.cuda(), lens.cuda(), codes, codes.clone(), steps, steps.clone(), query_start=start.cuda())
        for i, m in enumerate(fresh):
            c.append([i], upto, new[start[i]:start[i + 1]].float().numpy())
    assert pa.pa_get_device_status() == 0
    assert np.array_equal(codes.cpu().numpy(), c.codes) and np.array_equal(steps.cpu().numpy(), c.steps)
    return c, codes, steps


ENDS = [65248.0 + 32 * i for i in range(9)]          # the last nine numbers of fp16; the upper eight fill a frame's top code


@pytest.mark.parametrize("D", [64, 128])
def test_rows_read_back_finite(pa, D):
    H, B = 3, 16
    frames = ENDS + [65504.0] * 40
    firsts = [None] * len(ENDS) + [float(torch.tensor(0.37 * 1.31 ** i).half()) for i in range(40)]   # steps of all kinds, grown
    c, codes, steps = filled(frames, H, B, D, "f16", firsts)
    value = (c.codes.astype(np.float64) - 128) * c.steps.astype(np.float64)[..., None, None]
    assert (np.abs(value) >= 65520).any(axis=(1, 2, 3)).sum() > 8       # what rounding alone would make infinite
    slots = torch.arange(len(frames) * B, dtype=torch.int32).cuda()
    for dtype in ("f16", "bf16"):
        out = [torch.full((len(slots), H, D), float("nan"), dtype=TD[dtype], device="cuda") for _ in range(2)]
        pa.pa_cache_read_q8(codes, codes, steps, steps, slots, out[0], out[1])
        want = value.astype(np.float32).transpose(0, 2, 1, 3).reshape(-1, H, D)
        want = torch.from_numpy(largest_kept(want, dtype)).to(TD[dtype])
        for o in out:
            assert torch.isfinite(o).all() and torch.equal(o.cpu(), want)
    assert pa.pa_get_device_status() == 0


def test_what_fp16_does_not_hold_and_nan(pa):
    c, codes, steps = filled([1e9, 2.0 ** 60, 70000.0, 3.0], 1, 8, 64, "bf16", [None] * 4)
    steps[3] = float("nan")
    slots = torch.arange(32, dtype=torch.int32).cuda()
    k, v = (torch.empty(32, 1, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pa_cache_read_q8(codes, codes, steps, steps, slots, k, v)
    assert (k[:24].abs() == 65504).all() and (torch.sign(k[:24, 0, :3]).cpu() == torch.tensor([-1.0, 1.0, 1.0])).all()
    assert torch.isnan(k[24:]).all() and torch.equal(k[:24], v[:24])
    assert pa.pa_get_device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 4, 8, 16])
@pytest.mark.parametrize("window", [0, 40])
def test_decodes_stay_finite(pa, D, g, window):
    """Values of +-65504 everywhere: one token, several, a context in pieces that are joined, one in groups of pieces."""
    H, B, lens = 2, 16, [1, 30, 3000, 40000]
    gen = torch.Generator().manual_seed(g)
    tables, nb = paged(gen, lens, B)
    c, codes, steps = filled([65504.0] * 2, H, B, D, "f16", [None, 33.0])
    pick = torch.randint(0, 2, (nb,), generator=gen)
    codes, steps = codes[pick.cuda()].contiguous(), steps[pick.cuda()].contiguous()
    q = torch.randn(len(lens), H * g, D, generator=gen).half()
    zero = torch.full_like(codes, 128)                                  # keys: equal scores
    out = torch.full_like(q, float("nan"), device="cuda")
    n = torch.tensor(lens, dtype=torch.int32)
    pa.pa_decode_q8(q.cuda(), zero, codes, steps, steps, tables.cuda(), n.cuda(), 0.1, out, window=window)
    assert pa.pa_get_device_status() == 0
    for s, L in enumerate(lens):
        j = np.arange(max(0, L - window) if window else 0, L)
        f = pick[tables[s, j // B].long()].numpy()
        v = (c.codes[f, :, j % B].astype(np.float64) - 128) * c.steps[f].astype(np.float64)[..., None]
        ref = attend_seen(host64(q[s]), np.zeros_like(v), v, len(v) - 1, 0, 0, 0.1)
        tol = attention_tolerance(ref, torch.float16, host64(q[s]), np.zeros_like(v), v, 0.1, 2.0 ** -22)
        got = host64(out[s])
        assert np.isfinite(got).all() and (np.abs(got - largest_kept(ref, "f16")) <= tol).all(), (s, float(np.abs(got).max()))
    steps[int(tables[1, 1])] = float("nan")
    pa.pa_decode_q8(q.cuda(), zero, codes, steps, steps, tables.cuda(), n.cuda(), 0.1, out, window=window)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[[0, 2, 3]]).all()
