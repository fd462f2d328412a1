"""Frame bounds, the selection from them, and decode attention over the selected frames."""

import numpy as np
import pytest
import torch

from oracle.operators import attend, block_scores, select_blocks
from tests._operators_common import TD, attention_tolerance, host64, paged

pytestmark = pytest.mark.gpu


def make(lens, H, g, D, B, dtype, seed, poison=True):
    gen = torch.Generator().manual_seed(seed)
    tables, nb = paged(gen, lens, B)
    kc, vc = (torch.randn(nb, B, H, D, generator=gen).to(TD[dtype]) for _ in range(2))
    if poison:  # slots that hold no token
        live = torch.zeros(nb, B, dtype=torch.bool)
        for s, n in enumerate(lens):
            for j in range(-(-n // B)):
                live[tables[s, j], : n - j * B] = True
        kc[~live] = float("nan")
        vc[~live] = float("nan")
    q = torch.randn(len(lens), H * g, D, generator=gen).to(TD[dtype])
    return q.cuda(), kc.cuda(), vc.cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


def bounds_reference(kc, tables, lens, first, bounds):
    B = kc.shape[1]
    want = bounds.clone()
    for s, n in enumerate(lens.tolist()):
        for j in range(first[s] // B, -(-n // B)) if first[s] < n else ():
            f = int(tables[s, j])
            rows = kc[f, : min(B, n - j * B)]
            want[f, :, 0], want[f, :, 1] = rows.amin(0), rows.amax(0)
    return want


LENS = [0, 1, 7, 8, 9, 16, 31, 33, 100, 257, 1000]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,D,B", [(1, 64, 8), (3, 128, 16), (8, 128, 32), (2, 64, 256), (32, 128, 16)])
def test_bounds(pa, dtype, H, D, B):
    q, kc, vc, tables, lens = make(LENS, H, 1, D, B, dtype, H + B)
    old = torch.full((kc.shape[0], H, 2, D), 3.0, dtype=TD[dtype], device="cuda")
    for first in ([0] * len(LENS), [max(0, n - 1) for n in LENS], [n // 2 for n in LENS], [n for n in LENS], [n + 9 for n in LENS]):
        got = old.clone()
        pa.pa_block_bounds(kc, tables, lens, torch.tensor(first, dtype=torch.int32).cuda(), got)
        assert torch.equal(got, bounds_reference(kc, tables, lens, first, old))
    got = old.clone()
    pa.pa_block_bounds(kc, tables, lens, None, got)
    assert torch.equal(got, bounds_reference(kc, tables, lens, [0] * len(LENS), old))
    assert pa.pa_get_device_status() == 0


@pytest.mark.parametrize("H,most", [(5, 700), (1, 4000), (11, 300)])
def test_bounds_more_units_than_warps(pa, H, most):
    """Sequences of no, few and many frames: a warp's next frame is heads or several sequences further on."""
    g = torch.Generator().manual_seed(H)
    lens = [0, 1, 0, 0, 8, 9] + torch.randint(0, most, (90,), generator=g).tolist() + [3, 0, 0, 17, 0]
    q, kc, vc, tables, lens = make(lens, H, 1, 64, 8, "f16", H)
    old = torch.full((kc.shape[0], H, 2, 64), 3.0, dtype=torch.float16, device="cuda")
    for first in (torch.zeros(len(lens), dtype=torch.int32), (torch.rand(len(lens), generator=g) * 0.3 * lens.cpu()).to(torch.int32)):
        got = old.clone()
        pa.pa_block_bounds(kc, tables, lens, first.cuda(), got)
        assert torch.equal(got, bounds_reference(kc, tables, lens, first.tolist(), old))
    assert pa.pa_get_device_status() == 0


def test_bounds_bad_indexes(pa):
    q, kc, vc, tables, lens = make([100, 50, 40, 30], 2, 1, 64, 16, "f16", 1)
    old = torch.zeros(kc.shape[0], 2, 2, 64, dtype=torch.float16, device="cuda")
    bad_t, bad_l, first = tables.clone(), lens.clone(), torch.tensor([0, 0, 0, -1], dtype=torch.int32).cuda()
    bad_t[0, 2] = kc.shape[0]
    bad_l[1] = tables.shape[1] * 16 + 1
    got = old.clone()
    pa.pa_block_bounds(kc, bad_t, bad_l, first, got)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_BLOCK | pa.PA_DEV_BAD_LEN
    want = bounds_reference(kc, tables, lens, [0, 50, 0, 30], old)
    want[tables[0, 2].long()] = 0
    assert torch.equal(got, want)


def test_bounds_nan_keys(pa):
    q, kc, vc, tables, lens = make([32], 1, 1, 64, 16, "bf16", 2)
    f = int(tables[0, 0])
    kc[f, 3, 0, 5] = float("nan")
    kc[f, 0, 0, 6] = float("nan")
    b = torch.zeros(kc.shape[0], 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    pa.pa_block_bounds(kc, tables, lens, None, b)
    x = torch.nan_to_num(kc[f, :, 0].float(), nan=0.0)
    for d, skip in ((5, 3), (6, 0)):
        rest = torch.cat([x[:skip, d], x[skip + 1:, d]])
        assert float(b[f, 0, 0, d]) == float(rest.min()) and float(b[f, 0, 1, d]) == float(rest.max())


def with_bounds(pa, q, kc, tables, lens):
    b = torch.full((kc.shape[0], kc.shape[2], 2, kc.shape[3]), float("nan"), dtype=kc.dtype, device="cuda")
    pa.pa_block_bounds(kc, tables, lens, None, b)
    return b


def selection_reference(q, bounds, tables, lens, B, K, first, last):
    got = []
    for s, n in enumerate(lens.tolist()):
        f = tables[s, : -(-n // B)].long()
        sc = block_scores(q[s].float().cpu().numpy(), bounds[f].float().cpu().numpy())
        got.append(select_blocks(sc, K, first, last))
    return np.stack(got)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,g,D,B", [(1, 1, 64, 8), (3, 4, 128, 16), (2, 16, 128, 32), (4, 3, 64, 16), (2, 8, 128, 64)])
@pytest.mark.parametrize("K,first,last", [(1, 0, 0), (8, 1, 2), (5, 4, 4), (64, 1, 1), (300, 0, 1)])
def test_selection(pa, dtype, H, g, D, B, K, first, last):
    q, kc, vc, tables, lens = make(LENS + [3000, 2049], H, g, D, B, dtype, K + B)
    b = with_bounds(pa, q, kc, tables, lens)
    sel = torch.full((len(lens), H, K), -99, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(q, b, tables, lens, B, sel, keep_first=first, keep_last=last)
    assert pa.pa_get_device_status() == 0
    assert np.array_equal(sel.cpu().numpy(), selection_reference(q, b, tables, lens, B, K, first, last))


def test_selection_ties_and_strides(pa):
    """Frames of equal scores: the lower positions; lists as a slice of a wider tensor."""
    q, kc, vc, tables, lens = make([16 * 400], 2, 2, 64, 16, "f16", 5)
    kc[:] = 1.0
    kc[tables[0, 7].long()] = -1.0
    b = with_bounds(pa, q, kc, tables, lens)
    q.fill_(0.5)
    wide = torch.full((1, 3, 50), -99, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(q, b, tables, lens, 16, wide[:, :2, :40], keep_first=0, keep_last=0)
    assert wide[0, :2, :40].tolist() == [[j for j in range(41) if j != 7]] * 2
    assert (wide[:, 2] == -99).all() and (wide[:, :, 40:] == -99).all()


def test_selection_long_context(pa):
    """More frames than one block's threads, shared by few heads."""
    q, kc, vc, tables, lens = make([60000, 5], 1, 4, 64, 8, "bf16", 6)
    b = with_bounds(pa, q, kc, tables, lens)
    sel = torch.empty(2, 1, 100, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(q, b, tables, lens, 8, sel)
    assert np.array_equal(sel.cpu().numpy(), selection_reference(q, b, tables, lens, 8, 100, 1, 1))


@pytest.mark.parametrize("L,K", [(15000, 33), (30000, 700), (90000, 5), (160000, 64), (160000, 1)])
def test_selection_list_sizes(pa, L, K):
    """Lists for each number of threads, and one longer than the registers hold."""
    q, kc, vc, tables, lens = make([L, 400], 1, 2, 64, 8, "f16", K, poison=False)
    b = with_bounds(pa, q, kc, tables, lens)
    sel = torch.empty(2, 1, K, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(q, b, tables, lens, 8, sel, keep_first=1, keep_last=0)
    assert np.array_equal(sel.cpu().numpy(), selection_reference(q, b, tables, lens, 8, K, 1, 0))


def test_selection_scores_that_crowd(pa):
    """Nearly all scores in one corner of their range, many of them equal, and the last place among those."""
    q, kc, vc, tables, lens = make([8 * 1000], 1, 1, 64, 8, "bf16", 3, poison=False)
    b = torch.zeros(kc.shape[0], 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    q.fill_(1.0)
    f = tables[0].long()
    b[f, 0, 1, 0] = (torch.arange(1000, device="cuda") % 5).to(torch.bfloat16) * 2.0 ** -20
    b[f[17], 0, 1, 0] = 1e30
    b[f[23], 0, 1, 0] = -1e30
    for K in (1, 2, 150, 201, 202, 400, 999):
        sel = torch.empty(1, 1, K, dtype=torch.int32, device="cuda")
        pa.pa_select_blocks(q, b, tables, lens, 8, sel, keep_first=0, keep_last=0)
        assert np.array_equal(sel.cpu().numpy(), selection_reference(q, b, tables, lens, 8, K, 0, 0)), K


def test_selection_nan_scores_stay_inside(pa):
    """Non-finite scores rank somewhere: the list still holds distinct frames of the sequence."""
    q, kc, vc, tables, lens = make([8 * 500, 8 * 90], 2, 2, 64, 8, "f16", 4, poison=False)
    b = with_bounds(pa, q, kc, tables, lens)
    b[tables[0, ::3].long()] = float("nan")
    b[tables[0, 1::3].long()] = float("inf")
    b[tables[1, :90].long()] = float("nan")
    sel = torch.full((2, 2, 40), -9, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(q, b, tables, lens, 8, sel)
    assert pa.pa_get_device_status() == 0
    for s, n in enumerate((500, 90)):
        for h in range(2):
            x = sel[s, h].tolist()
            assert x == sorted(set(x)) and 0 <= x[0] and x[-1] < n and x[0] == 0 and x[-1] == n - 1


def test_selection_bad_indexes(pa):
    q, kc, vc, tables, lens = make([320, 320, 320], 2, 2, 64, 16, "f16", 7)
    b = with_bounds(pa, q, kc, tables, lens)
    sel, good = (torch.full((3, 2, 6), -99, dtype=torch.int32, device="cuda") for _ in range(2))
    pa.pa_select_blocks(q, b, tables, lens, 16, good)
    bad_t, bad_l = tables.clone(), lens.clone()
    bad_t[0, 10] = -3
    bad_l[1] = 321
    pa.pa_select_blocks(q, b, bad_t, bad_l, 16, sel)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_BLOCK | pa.PA_DEV_BAD_LEN
    assert torch.equal(sel[2], good[2])
    assert (sel[1] == -1).all()
    assert (sel[0] != 10).all() and (sel[0] >= 0).all()


# ---- decode over listed frames ---------------------------------------------------------------------------
def check_selected(pa, case, sel, scale, dtype):
    q, kc, vc, tables, lens = case
    out = torch.full_like(q, float("nan"))
    pa.pa_decode_selected(q, kc, vc, tables, lens, sel, scale, out)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == 0
    compare_selected(out, case, sel, scale, dtype)
    return out


def compare_selected(out, case, sel, scale, dtype, only=None):
    """out against 64 bits; only: the (sequence, key head) pairs looked at."""
    q, kc, vc, tables, lens = case
    B, H = kc.shape[1], kc.shape[2]
    g = q.shape[1] // H
    got, qh = host64(out), host64(q)
    kh, vh, th = kc.cpu(), vc.cpu(), tables.cpu().long()
    for s, n in enumerate(lens.tolist()):
        for h in range(H):
            if only is not None and (s, h) not in only:
                continue
            tok = []
            for e in sel[s, h].tolist()[: -(-n // B)]:
                if e == -1:
                    break
                tok += [(int(th[s, e]), i) for i in range(min(B, n - e * B))]
            f, i = torch.tensor([t[0] for t in tok]).long(), torch.tensor([t[1] for t in tok]).long()
            k, v = (host64(c[f, i, h])[:, None] if len(tok) else np.zeros((0, 1, q.shape[2])) for c in (kh, vh))
            ref = attend(qh[s, h * g:h * g + g], k, v, scale)
            tol = attention_tolerance(ref, TD[dtype], qh[s, h * g:h * g + g], k, v, scale, 2.0 ** (-22 if dtype == "f16" else -16))
            err = np.abs(got[s, h * g:h * g + g] - ref)
            assert (err <= tol).all(), (s, h, n, float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,g,D,B", [(1, 1, 64, 8), (3, 4, 128, 16), (2, 16, 128, 32), (4, 3, 64, 16), (2, 8, 128, 64), (1, 5, 128, 256),
                                     (2, 2, 128, 8), (8, 1, 128, 16)])
@pytest.mark.parametrize("K", [1, 7, 40])
def test_selected_decode(pa, dtype, H, g, D, B, K):
    case = make(LENS + [2049], H, g, D, B, dtype, K + B)
    q, kc, vc, tables, lens = case
    sel = torch.empty(len(lens), H, K, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(q, with_bounds(pa, q, kc, tables, lens), tables, lens, B, sel, keep_first=1, keep_last=1)
    check_selected(pa, case, sel, D ** -0.5, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_selected_decode_any_order(pa, dtype):
    """Lists in any order (the last, partly filled frame among the first), ended early, empty, with a frame listed twice."""
    for B in (8, 16, 64):
        case = make([1000, 999, 100, 50], 2, 4, 128, B, dtype, B)
        n = [-(-x // B) for x in (1000, 999, 100, 50)]
        sel = torch.full((4, 2, 9), -1, dtype=torch.int32)
        sel[0, 0] = torch.tensor([n[0] - 1, 0, 5, 3, 2, 9, 8, 1, 4])
        sel[0, 1, :4] = torch.tensor([7, n[0] - 1, 6, 0])
        sel[1, 0, :3] = torch.tensor([4, 4, 1])
        sel[2, 0, :2] = torch.tensor([n[2] - 1, 0])
        sel[2, 1, 4:] = 0                                   # behind the end: not read
        sel[3, :, 0] = n[3] - 1
        check_selected(pa, case, sel.cuda(), 0.09, dtype)


@pytest.mark.parametrize("g", [1, 4, 16])
def test_selected_decode_long_lists(pa, g):
    """Lists cut into many pieces (joined in groups) beside short ones."""
    case = make([64 * 500, 64 * 3, 0], 1, g, 64, 64, "bf16", g)
    sel = torch.full((3, 1, 500), -1, dtype=torch.int32)
    sel[0, 0] = torch.randperm(500, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    sel[1, 0, :2] = torch.tensor([2, 0])
    check_selected(pa, case, sel.cuda(), 0.125, "bf16")


def test_every_frame_selected_is_pa_decode(pa):
    """All frames listed: the plain decode's result, to both calls' tolerances."""
    q, kc, vc, tables, lens = make([300, 17, 1, 64], 4, 1, 128, 16, "f16", 9)
    K = tables.shape[1]
    sel = torch.empty(4, 4, K, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(q, with_bounds(pa, q, kc, tables, lens), tables, lens, 16, sel)
    out, ref = torch.empty_like(q), torch.empty_like(q)
    pa.pa_decode_selected(q, kc, vc, tables, lens, sel, 0.09, out)
    pa.pa_decode(q, kc, vc, tables, lens, 0.09, ref)
    assert (out.float() - ref.float()).abs().max() <= 2e-3


def test_selected_decode_bad_indexes(pa):
    case = make([320, 320, 320, 320], 2, 2, 64, 16, "bf16", 11)
    q, kc, vc, tables, lens = case
    sel = torch.arange(4, dtype=torch.int32).repeat(4, 2, 1).cuda()
    good = check_selected(pa, case, sel, 0.1, "bf16")
    bad_t, bad_l, bad_s = tables.clone(), lens.clone(), sel.clone()
    bad_t[0, 2] = kc.shape[0]
    bad_l[1] = -4
    bad_s[2, 1, 3] = 20
    bad_s[3, 0, 0] = -2
    out = torch.full_like(q, float("nan"))
    pa.pa_decode_selected(q, kc, vc, bad_t, bad_l, bad_s, 0.1, out)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_BLOCK | pa.PA_DEV_BAD_LEN
    assert not out[0].any() and not out[1].any() and not out[2, 2:].any() and not out[3, :2].any()
    # the batch is cut among the warps by its lengths: with one of them bad the cuts lie elsewhere and the other
    # heads' fp32 sums are taken in another order, so they are held to the 64-bit result and not to equal bits
    compare_selected(out, case, sel, 0.1, "bf16", only={(2, 0), (3, 1)})
    assert torch.equal(check_selected(pa, case, sel, 0.1, "bf16"), good)


def test_selected_decode_frames_behind_4_gib(pa):
    H, D, B = 8, 128, 16
    nb = 140_000
    q, kc, vc, tables, lens = make([70, 33], H, 4, D, B, "f16", 13, poison=False)
    n = kc.shape[0]
    big = [torch.empty(nb, B, H, D, dtype=torch.float16, device="cuda") for _ in range(2)]
    for x, c in zip(big, (kc, vc)):
        x[nb - n:] = c
    far = torch.where(tables >= 0, tables + (nb - n), tables)
    bounds = torch.empty(nb, H, 2, D, dtype=torch.float16, device="cuda")
    pa.pa_block_bounds(big[0], far, lens, None, bounds)
    near = with_bounds(pa, q, kc, tables, lens)
    live = tables[tables >= 0].long()
    assert torch.equal(bounds[live + (nb - n)], near[live])
    sel, sel2 = (torch.empty(2, H, 3, dtype=torch.int32, device="cuda") for _ in range(2))
    pa.pa_select_blocks(q, bounds, far, lens, B, sel)
    pa.pa_select_blocks(q, near, tables, lens, B, sel2)
    assert torch.equal(sel, sel2)
    out, ref = torch.empty_like(q), torch.empty_like(q)
    pa.pa_decode_selected(q, big[0], big[1], far, lens, sel, 0.1, out)
    pa.pa_decode_selected(q, kc, vc, tables, lens, sel, 0.1, ref)
    assert torch.equal(out, ref)
    assert pa.pa_get_device_status() == 0


def test_empty_batches(pa):
    q, kc, vc, tables, lens = make([0, 0], 2, 2, 64, 16, "f16", 14)
    none = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    b = torch.zeros(kc.shape[0], 2, 2, 64, dtype=torch.float16, device="cuda")
    for t in (tables, none):
        pa.pa_block_bounds(kc, t, lens, None, b)
        assert not b.any()
        sel = torch.full((2, 2, 3), 5, dtype=torch.int32, device="cuda")
        pa.pa_select_blocks(q, b, t, lens, 16, sel)
        assert (sel == -1).all()
        out = torch.full_like(q, float("nan"))
        pa.pa_decode_selected(q, kc, vc, t, lens, sel, 0.1, out)
        assert not out.any()
    n = pa.pa_launch_count()
    pa.pa_decode_selected(q[:0], kc, vc, tables[:0], lens[:0], sel[:0], 0.1, out[:0])
    pa.pa_select_blocks(q[:0], b, tables[:0], lens[:0], 16, sel[:0])
    pa.pa_block_bounds(kc, tables[:0], lens[:0], None, b)
    assert pa.pa_launch_count() == n
    assert pa.pa_get_device_status() == 0
