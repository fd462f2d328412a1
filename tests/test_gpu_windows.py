"""Attention over a window and the first tokens: single queries and chunks of queries, against the 64-bit oracle (GPU)."""

import numpy as np
import pytest
import torch

from oracle.windows import attend_seen
from tests._operators_common import TD, attention_tolerance, host64
from tests._windows_common import hidden_slots, window_tables

pytestmark = pytest.mark.gpu


# ---- single queries ------------------------------------------------------------------------------------
def decode_case(lens, H, g, D, B, dtype, window, sinks, seed, q_scale=1.0, poison=True):
    gen = torch.Generator().manual_seed(seed)
    one = [1] * len(lens)
    tables, nb = window_tables(gen, lens, one, B, window, sinks, gone=10 ** 9)   # never to be read
    kc, vc = (torch.randn(nb, B, H, D, generator=gen).to(TD[dtype]) for _ in range(2))
    if poison:
        hide = hidden_slots(lens, one, B, window, sinks, tables, nb)
        kc[hide], vc[hide] = float("nan"), float("nan")
    q = (torch.randn(len(lens), H * g, D, generator=gen) * q_scale).to(TD[dtype])
    return q, kc, vc, tables, torch.tensor(lens, dtype=torch.int32)


def weight_step(dtype):
    return 2.0 ** (-22 if dtype == "f16" else -16)                     # two parts of the cache's type


def reference(case, window, sinks, scale, s):
    q, kc, vc, tables, lens = case
    B, n = kc.shape[1], int(lens[s])
    j = torch.arange(n)
    j = j[(j >= n - window) | (j < sinks)]
    f = tables[s, j // B].long()
    k, v = host64(kc[f, j % B]), host64(vc[f, j % B])
    return attend_seen(host64(q[s]), k, v, len(k) - 1, 0, 0, scale), k, v


def check_decode(pa, case, window, sinks, scale, dtype, seqs=None, stream=None):
    q, kc, vc, tables, lens = case
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    pa.pa_decode_window(q.cuda(), kc.cuda(), vc.cuda(), tables.cuda(), lens.cuda(), window, scale, out, sinks=sinks)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == 0
    got = host64(out)
    for s in range(len(lens)) if seqs is None else seqs:
        ref, k, v = reference(case, window, sinks, scale, s)
        tol = attention_tolerance(ref, TD[dtype], host64(q[s]), k, v, scale, weight_step(dtype))
        err = np.abs(got[s] - ref)
        assert (err <= tol).all(), (s, int(lens[s]), float((err - tol).max()), float(err.max()))
    return out


LENS = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 64, 100, 255, 257, 700]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (7, 1), (16, 16), (20, 0), (33, 17), (100, 4), (256, 100), (10000, 3)])
@pytest.mark.parametrize("B", [8, 16, 32, 256])
@pytest.mark.parametrize("dtype,D,H,g", [("f16", 128, 2, 4), ("bf16", 64, 3, 1), ("bf16", 128, 1, 7), ("f16", 64, 1, 16)])
def test_decode_lengths(pa, dtype, D, H, g, B, window, sinks):
    check_decode(pa, decode_case(LENS, H, g, D, B, dtype, window, sinks, B + window), window, sinks, D ** -0.5, dtype)


def test_decode_widest_window_and_most_sinks(pa):
    big = 2 ** 31 - 1
    case = decode_case(LENS, 2, 2, 64, 16, "f16", 10 ** 6, 0, 1)
    full = check_decode(pa, case, big, 0, 0.1, "f16")
    assert torch.equal(full, check_decode(pa, case, big, big, 0.1, "f16"))
    assert torch.equal(full, check_decode(pa, case, 1, big, 0.1, "f16"))
    assert torch.equal(full, check_decode(pa, case, 3, 700, 0.1, "f16"))


@pytest.mark.parametrize("g", [1, 4, 8])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_split_windows(pa, g, dtype):
    """Few heads and wide windows: pieces of one joined, short sequences beside it."""
    case = decode_case([40000, 3, 0, 5000, 1], 1, g, 128, 16, dtype, 12345, 70, 3)
    check_decode(pa, case, 12345, 70, 128 ** -0.5, dtype)


def test_decode_many_sequences(pa):
    lens = [(i * 7) % 150 for i in range(1000)]
    case = decode_case(lens, 4, 2, 64, 16, "bf16", 40, 5, 4)
    check_decode(pa, case, 40, 5, 0.125, "bf16", seqs=range(0, 1000, 37))


@pytest.mark.parametrize("scale", [0.0, -0.3, 5.0])
def test_decode_scales(pa, scale):
    case = decode_case([500, 17, 64], 2, 4, 128, 16, "f16", 100, 4, 6)
    check_decode(pa, case, 100, 4, scale, "f16")


def test_decode_equals_pa_decode_over_whole_sequences(pa):
    """Where every token is attended, the result is pa_decode's within both calls' tolerances."""
    case = decode_case([300, 41], 8, 1, 128, 16, "f16", 10 ** 6, 0, 7, poison=False)
    q, kc, vc, tables, lens = (x.cuda() for x in case)
    out = check_decode(pa, case, 300, 0, 0.1, "f16")
    ref = torch.empty_like(q)
    pa.pa_decode(q, kc, vc, tables, lens, 0.1, ref)
    assert (out.float() - ref.float()).abs().max() <= 2e-3


def test_decode_rows_in_descending_scores(pa):
    for sign in (1, -1):
        q, kc, vc, tables, n = decode_case([900], 1, 1, 128, 16, "f16", 640, 20, 9)
        k = torch.zeros(900, 128)
        k[:, 0] = sign * torch.arange(900) * 0.5
        for j in range(57):
            f = int(tables[0, j])
            if f < kc.shape[0]:
                kc[f, : min(16, 900 - 16 * j), 0] = k[16 * j:16 * j + 16].half()
        q.zero_()
        q[0, 0, 0] = 8.0
        check_decode(pa, (q, kc, vc, tables, n), 640, 20, 0.5, "f16")


def test_decode_bad_indexes(pa):
    window, sinks = 20, 3
    q, kc, vc, tables, lens = decode_case([100, 50, 40, 30], 2, 4, 64, 16, "f16", window, sinks, 10)
    check_decode(pa, (q, kc, vc, tables, lens), window, sinks, 0.125, "f16")
    bad_t, bad_l = tables.clone(), lens.clone()
    bad_t[0, 0] = kc.shape[0]                                          # its sinks' frame
    bad_t[1, 3] = -5                                                   # its last frame
    bad_l[2] = tables.shape[1] * 16 + 1
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    pa.pa_decode_window(q.cuda(), kc.cuda(), vc.cuda(), bad_t.cuda(), bad_l.cuda(), window, 0.125, out, sinks=sinks)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_BLOCK | pa.PA_DEV_BAD_LEN
    assert not out[:3].any()
    ref, k, v = reference((q, kc, vc, tables, lens), window, sinks, 0.125, 3)
    assert (np.abs(host64(out[3]) - ref) <= attention_tolerance(ref, torch.float16, host64(q[3]), k, v, 0.125, 2.0 ** -22)).all()
    check_decode(pa, (q, kc, vc, tables, lens), window, sinks, 0.125, "f16")   # later calls start clean


def test_decode_strided_rows_and_tables(pa):
    q, kc, vc, tables, lens = decode_case([100, 50, 40], 2, 4, 128, 16, "bf16", 30, 2, 12)
    ref = check_decode(pa, (q, kc, vc, tables, lens), 30, 2, 0.1, "bf16")
    wide_q = torch.full((3, 8 * 128 + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_q[:, : 8 * 128] = q.flatten(1).cuda()
    wide_o = torch.full((3, 8 * 128 + 32), 9.0, dtype=torch.bfloat16, device="cuda")
    wide_t = torch.full((3, 40), -7, dtype=torch.int32, device="cuda")
    wide_t[:, : tables.shape[1]] = tables.cuda()
    pa.pa_decode_window(wide_q[:, : 8 * 128].view(3, 8, 128), kc.cuda(), vc.cuda(), wide_t[:, : tables.shape[1]], lens.cuda(), 30, 0.1,
                        wide_o[:, : 8 * 128].view(3, 8, 128), sinks=2)
    assert torch.equal(wide_o[:, : 8 * 128].reshape(3, 8, 128), ref)
    assert (wide_o[:, 8 * 128:] == 9).all()


def test_decode_empty_batches_and_no_columns(pa):
    q, kc, vc, tables, lens = decode_case([0, 0, 0], 2, 1, 64, 16, "f16", 5, 1, 14)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    none = torch.empty(3, 0, dtype=torch.int32, device="cuda")
    pa.pa_decode_window(q.cuda(), kc.cuda(), vc.cuda(), none, lens.cuda(), 5, 0.1, out, sinks=1)
    assert not out.any()
    n = pa.pa_launch_count()
    pa.pa_decode_window(q[:0].cuda(), kc.cuda(), vc.cuda(), tables[:0].cuda(), lens[:0].cuda(), 5, 0.1, out[:0])
    assert pa.pa_launch_count() == n
    assert pa.pa_get_device_status() == 0


def test_decode_table_of_almost_2_31_tokens(pa):
    """One sequence of 2^31 - 1 tokens whose table repeats a few frames: positions next to int32's end."""
    B, blocks = 8, 2 ** 28 - 1
    L = blocks * B
    gen = torch.Generator().manual_seed(20)
    kc, vc = (torch.randn(4, B, 1, 64, generator=gen).half() for _ in range(2))
    t = torch.full((1, blocks), -1, dtype=torch.int32, device="cuda")
    t[0, 0], t[0, -3:] = 3, torch.tensor([1, 0, 2], dtype=torch.int32)
    q = torch.randn(1, 2, 64, generator=gen).half()
    out = torch.empty_like(q, device="cuda")
    n = torch.tensor([L], dtype=torch.int32, device="cuda")
    pa.pa_decode_window(q.cuda(), kc.cuda(), vc.cuda(), t, n, 19, 0.125, out, sinks=5)
    assert pa.pa_get_device_status() == 0
    k, v = (torch.cat([c[3, :5], c[1, -3:], c[0], c[2]]) for c in (kc, vc))
    ref = attend_seen(host64(q[0]), host64(k), host64(v), len(k) - 1, 0, 0, 0.125)
    tol = attention_tolerance(ref, torch.float16, host64(q[0]), host64(k), host64(v), 0.125, 2.0 ** -22)
    assert (np.abs(host64(out[0]) - ref) <= tol).all()


def test_decode_same_bits_every_time(pa):
    q, kc, vc, tables, lens = (x.cuda() for x in decode_case([9000, 40, 777, 2048], 2, 4, 128, 32, "bf16", 1500, 4, 15))
    first = torch.empty_like(q)
    pa.pa_decode_window(q, kc, vc, tables, lens, 1500, 0.1, first, sinks=4)
    for _ in range(20):
        again = torch.empty_like(q)
        pa.pa_decode_window(q, kc, vc, tables, lens, 1500, 0.1, again, sinks=4)
        assert torch.equal(first, again)


# ---- chunks of queries ---------------------------------------------------------------------------------
def chunk_case(lens, fresh, H, g, B, dtype, window, sinks, seed, q_scale=1.0, spare_rows=0):
    gen = torch.Generator().manual_seed(seed)
    tables, nb = window_tables(gen, lens, fresh, B, window, sinks, gone=-1)
    kc, vc = (torch.randn(nb, B, H, 128, generator=gen).to(TD[dtype]) for _ in range(2))
    start = torch.tensor([0] + list(np.cumsum(fresh)), dtype=torch.int32)
    q = (torch.randn(int(start[-1]) + spare_rows, H * g, 128, generator=gen) * q_scale).to(TD[dtype])
    return q, kc, vc, tables, torch.tensor(lens, dtype=torch.int32), start


def chunk_tolerance(ref, dtype, q, k, v, scale):
    """attention_tolerance, and the weights as pa_prefill carries them: in fp16 one part, off by 2^-11 of itself, a small one
    by half of fp16's least number, 2^-25 of the reference; bf16 has two parts."""
    step = 2.0 ** -11 + len(k) * 2.0 ** -25 if dtype == "f16" else 2.0 ** -16
    return attention_tolerance(ref, TD[dtype], q, k, v, scale, step)


def check_chunk(pa, case, window, sinks, scale, dtype, rows=None):
    q, kc, vc, tables, lens, start = case
    B = kc.shape[1]
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    pa.pa_prefill_window(q.cuda(), kc.cuda(), vc.cuda(), tables.cuda(), lens.cuda(), start.cuda(), window, scale, out, sinks=sinks)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == 0
    got = host64(out)
    for s in range(len(lens)):
        n, r0, r1 = int(lens[s]), int(start[s]), int(start[s + 1])
        lo = max(0, n - (r1 - r0) + 1 - window)
        j = torch.arange(n)
        j = j[(j >= lo) | (j < sinks)]
        f = tables[s, j // B].long()
        k, v, j = host64(kc[f, j % B]), host64(vc[f, j % B]), j.numpy()
        for r in range(r0, r1) if rows is None else [x for x in rows if r0 <= x < r1]:
            p = n - (r1 - r0) + r - r0
            on = (j <= p) & ((j > p - window) | (j < sinks))
            ref = attend_seen(host64(q[r]), k[on], v[on], int(on.sum()) - 1, 0, 0, scale)
            tol = chunk_tolerance(ref, dtype, host64(q[r]), k[on], v[on], scale)
            err = np.abs(got[r] - ref)
            assert (err <= tol).all(), (s, r, p, float((err - tol).max()), float(err.max()))
    assert (got[int(start[-1]):] == 7).all()                           # rows behind the last sequence
    return out


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (5, 0), (64, 70), (100, 4), (128, 0), (129, 130), (300, 1), (100000, 9)])
@pytest.mark.parametrize("dtype,H,g,B", [("f16", 2, 1, 16), ("bf16", 1, 4, 32), ("f16", 1, 3, 8), ("bf16", 2, 1, 128), ("f16", 1, 16, 64)])
def test_chunk_lengths(pa, dtype, H, g, B, window, sinks):
    fresh = [1, 0, 2, 130, 64, 257, 1, 300]
    lens = [1, 0, 9, 130, 700, 500, 400, 1234]
    case = chunk_case(lens, fresh, H, g, B, dtype, window, sinks, window + B, spare_rows=3)
    rows = list(range(0, 6)) + list(range(120, 140)) + list(range(190, 200, 3)) + list(range(440, 470, 5)) + list(range(640, 755, 19)) + [754]
    check_chunk(pa, case, window, sinks, 128 ** -0.5, dtype, rows)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 30), (128, 0), (150, 7), (300, 130), (100000, 9)])
@pytest.mark.parametrize("dtype,H,g,B", [("f16", 16, 1, 16), ("bf16", 5, 3, 8), ("bf16", 4, 4, 32), ("f16", 3, 6, 128)])
def test_chunk_of_many_heads(pa, dtype, H, g, B, window, sinks):
    """More tiles than thread blocks: two tiles of a head a block, or a tile of two heads where they share a key head."""
    fresh = [1, 0, 2, 130, 64, 257, 1, 300]
    lens = [1, 0, 9, 130, 700, 500, 400, 1234]
    case = chunk_case(lens, fresh, H, g, B, dtype, window, sinks, window + B, spare_rows=3)
    check_chunk(pa, case, window, sinks, 128 ** -0.5, dtype, [0, 1, 2, 3, 131, 132, 133, 196, 197, 324, 325, 400, 453, 454, 455, 581, 582, 700, 754])


@pytest.mark.parametrize("lens,fresh", [([5], [5]), ([128], [128]), ([129], [129]), ([256], [1]), ([257], [200]), ([384], [384]), ([513], [513])])
def test_chunk_of_few_tiles(pa, lens, fresh):
    """One tile a block, its key tiles to two slots in turn: one, two, odd and even numbers of them."""
    for window, sinks in ((10 ** 6, 0), (200, 3), (1, 0), (130, 0)):
        case = chunk_case(lens, fresh, 1, 2, 16, "bf16", window, sinks, lens[0] + window)
        check_chunk(pa, case, window, sinks, 0.09, "bf16", list(range(0, fresh[0], 17)) + [fresh[0] - 1])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_chunk_of_a_whole_prompt(pa, dtype):
    case = chunk_case([1500], [1500], 1, 2, 16, dtype, 200, 10, 3)
    check_chunk(pa, case, 200, 10, 128 ** -0.5, dtype, range(0, 1500, 23))


def test_chunk_with_a_window_over_everything_is_prefill(pa):
    # more tiles than thread blocks and a query head a key head: the slots are those of pa_prefill
    q, kc, vc, tables, lens, start = (x.cuda() for x in chunk_case([300, 500], [300, 77], 60, 1, 16, "f16", 10 ** 6, 0, 4))
    a, b = torch.empty_like(q), torch.empty_like(q)
    pa.pa_prefill_window(q, kc, vc, tables, lens, start, 2 ** 31 - 1, 0.1, a, sinks=2 ** 31 - 1)
    pa.pa_prefill(q, kc, vc, tables, lens, start, 0.1, b)
    assert torch.equal(a, b)
    pa.pa_prefill_window(q, kc, vc, tables, lens, start, 1, 0.1, a, sinks=500)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_chunk_scores_that_rise_and_fall(pa, dtype):
    """Sharp scores, each key far above or below the one before: the reference moves at every tile, and the window leaves the largest behind."""
    for sign in (1, -1):
        q, kc, vc, tables, lens, start = chunk_case([900], [400], 1, 1, 16, dtype, 150, 5, 5)
        k = torch.zeros(900, 128)
        k[:, 0] = sign * torch.arange(900) * 0.25
        for j in range(57):
            f = int(tables[0, j])
            if f >= 0:
                kc[f, : min(16, 900 - 16 * j), 0] = k[16 * j:16 * j + 16].to(TD[dtype])
        q.zero_()
        q[:, 0, 0] = 8.0
        check_chunk(pa, (q, kc, vc, tables, lens, start), 150, 5, 0.5, dtype, range(0, 400, 7))


def test_chunk_last_row_equals_the_single_query(pa):
    """A chunk's last query and pa_decode_window of the same one attend the same tokens."""
    case = chunk_case([700, 90], [130, 1], 2, 4, 16, "bf16", 100, 4, 6)
    q, kc, vc, tables, lens, start = (x.cuda() for x in case)
    out = check_chunk(pa, case, 100, 4, 0.09, "bf16", [129, 130])
    one = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    last = start[1:].long() - 1
    pa.pa_decode_window(q[last].contiguous(), kc, vc, tables, lens, 100, 0.09, one, sinks=4)
    assert (one.float() - out[last].float()).abs().max() <= 2.0 ** -7 * one.float().abs().max()   # a step of bf16 each


def test_chunk_bad_indexes(pa):
    window, sinks = 50, 20
    q, kc, vc, tables, lens, start = chunk_case([200, 300, 100, 64], [40, 33, 50, 64], 1, 2, 16, "f16", window, sinks, 7)
    good = check_chunk(pa, (q, kc, vc, tables, lens, start), window, sinks, 0.1, "f16", [0, 39, 40, 72, 73, 122, 123, 186])
    bad_l, bad_t = lens.clone(), tables.clone()
    bad_l[1] = 32                                                      # fewer tokens than queries
    out = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
    pa.pa_prefill_window(q.cuda(), kc.cuda(), vc.cuda(), tables.cuda(), bad_l.cuda(), start.cuda(), window, 0.1, out, sinks=sinks)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_LEN
    assert (out[40:73] == 5).all() and torch.equal(out[:40], good[:40]) and torch.equal(out[73:], good[73:])
    bad_t[2, 6] = kc.shape[0]                                          # the frame of tokens 96 .. 99
    pa.pa_prefill_window(q.cuda(), kc.cuda(), vc.cuda(), bad_t.cuda(), lens.cuda(), start.cuda(), window, 0.1, out, sinks=sinks)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_BLOCK
    assert torch.equal(out[:73], good[:73]) and torch.equal(out[73 + 46 - 30:73 + 46], good[73 + 46 - 30:73 + 46])


def test_chunk_more_sequences_than_a_launch_holds(pa):
    S = 9000
    lens = [1 + i % 40 for i in range(S)]
    case = chunk_case(lens, [1] * S, 1, 1, 8, "f16", 10, 2, 8)
    check_chunk(pa, case, 10, 2, 0.1, "f16", range(0, S, 401))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [3, 5, 8, 12, 16])
def test_decode_joins_of_many_queries(pa, g, D):
    """A window of 12345 tokens is joined in groups; of 400 windows of 260 tokens most are in pieces, and a block joins several."""
    check_decode(pa, decode_case([40000, 3, 0, 5000, 1], 1, g, D, 16, "f16", 12345, 70, 30 + g), 12345, 70, D ** -0.5, "f16")
    check_decode(pa, decode_case([300 - i % 7 for i in range(200)], 2, g, D, 16, "bf16", 256, 4, 31 + g), 256, 4, D ** -0.5, "bf16", seqs=range(0, 200, 3))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,g", [(40, 1), (20, 3), (20, 2), (5, 16)])
def test_chunk_tiles_of_many_heads_with_windows_and_sinks_inside(pa, dtype, H, g):
    """Items of both slots, one after another in a block, whose windows begin and sinks end inside a tile."""
    case = chunk_case([900, 301, 5], [390, 131, 5], H, g, 16, dtype, 333, 21, 7)
    check_chunk(pa, case, 333, 21, 128 ** -0.5, dtype, list(range(0, 390, 41)) + list(range(391, 526, 17)))
