"""NaN and infinities in the queries and keys of query chunks over windows: a query that attends one has a row of NaN, as a single query has,
and every other row its bits of before (GPU)."""

import pytest
import torch

from tests.test_gpu_windows import chunk_case

pytestmark = pytest.mark.gpu

# two tiles of a head a block (an odd number of queries a key head), a tile of two heads (even), key tiles to two slots (few tiles)
KINDS = [(40, 1), (20, 2), (1, 2)]


def run(pa, case, window, sinks):
    q, kc, vc, tables, lens, start = (x.cuda() for x in case)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    pa.pa_prefill_window(q, kc, vc, tables, lens, start, window, 0.09, out, sinks=sinks)
    assert pa.pa_get_device_status() == 0
    return out


def single(pa, case, window, sinks, row):
    """pa_decode_window of sequence 0's query in `row`, over the tokens up to its own."""
    q, kc, vc, tables, lens, start = (x.cuda() for x in case)
    upto = lens[:1] - int(start[1]) + row + 1
    one = torch.empty(1, *q.shape[1:], dtype=q.dtype, device="cuda")
    pa.pa_decode_window(q[row:row + 1].contiguous(), kc, vc, tables[:1], upto, window, 0.09, one, sinks=sinks)
    assert pa.pa_get_device_status() == 0
    return one[0]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,g", KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_queries(pa, dtype, H, g, bad):
    window, sinks = 150, 5
    case = chunk_case([700, 90], [300, 60], H, g, 16, dtype, window, sinks, 1)
    clean = run(pa, case, window, sinks)
    rows = torch.tensor([0, 3, 127, 128, 200, 255, 299, 310])
    case[0][rows, 0, 7] = bad
    out = run(pa, case, window, sinks)
    hit = torch.zeros(len(out), H * g, dtype=torch.bool, device="cuda")
    hit[rows.cuda(), 0] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])
    assert torch.isnan(single(pa, case, window, sinks, 200)[0]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,g", KINDS)
@pytest.mark.parametrize("at", [2, 4, 430, 511, 512, 699])              # positions: sinks, under the window of some queries, the last
def test_keys(pa, dtype, H, g, at):
    window, sinks, n, c = 150, 5, 700, 300
    case = chunk_case([n, 90], [c, 60], H, g, 16, dtype, window, sinks, 2)
    clean = run(pa, case, window, sinks)
    case[1][int(case[3][0, at // 16]), at % 16, H - 1, 9] = float("nan")
    out = run(pa, case, window, sinks)
    p = torch.arange(n - c, n)
    seen = (at <= p) & ((at > p - window) | (at < sinks))
    hit = torch.zeros(len(out), H * g, dtype=torch.bool, device="cuda")
    hit[: c, (H - 1) * g:] = seen.cuda()[:, None]
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])
    for row in (0, 130, 299):
        assert torch.isnan(single(pa, case, window, sinks, row)[H * g - 1]).all() == bool(seen[row])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,g", KINDS)
def test_keys_that_no_query_sees_may_hold_anything(pa, dtype, H, g):
    """Keys, not values: behind the sequence's end, beside the sinks, before the window of the first query."""
    from tests._windows_common import hidden_slots

    window, sinks, lens, fresh = 150, 5, [700, 90], [300, 60]
    case = chunk_case(lens, fresh, H, g, 16, dtype, window, sinks, 3)
    clean = run(pa, case, window, sinks)
    hide = hidden_slots(lens, fresh, 16, window, sinks, case[3], case[1].shape[0])
    case[1][hide] = float("nan")
    assert torch.equal(run(pa, case, window, sinks), clean)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,g", KINDS)
def test_rows_whose_scores_are_all_minus_infinity(pa, dtype, H, g):
    window, sinks = 150, 5
    case = chunk_case([700, 90], [300, 60], H, g, 16, dtype, window, sinks, 4)
    case[0][..., 0] = 1.0
    case[1][..., 0] = float("-inf")
    out = run(pa, case, window, sinks)
    assert not out.any() and not single(pa, case, window, sinks, 200).any()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,g", KINDS)
def test_values(pa, dtype, H, g):
    """A value that is not finite reaches that element of the rows that attend it, perhaps of others of its sequence and head, and
    nothing else."""
    window, sinks, n, c, at = 150, 5, 700, 300, 512
    case = chunk_case([n, 90], [c, 60], H, g, 16, dtype, window, sinks, 5)
    clean = run(pa, case, window, sinks)
    case[2][int(case[3][0, at // 16]), at % 16, 0, 9] = float("inf")
    out = run(pa, case, window, sinks)
    p = torch.arange(n - c, n)
    seen = (at <= p) & (at > p - window)
    assert not torch.isfinite(out[: c, : g, 9][seen.cuda()]).any()
    keep = torch.ones(out.shape, dtype=torch.bool, device="cuda")
    keep[: c, : g, 9] = False
    assert torch.equal(out[keep], clean[keep])
