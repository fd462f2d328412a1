"""The 8-bit cache: its bytes and steps, its values read back, and decode attention over it (GPU)."""

import numpy as np
import pytest
import torch

from oracle.windows import Cache8, attend_seen, seen
from tests._operators_common import TD, attention_tolerance, host64, paged
from tests._windows_common import cache8, on_gpu, window_tables

pytestmark = pytest.mark.gpu


# ---- append and read -----------------------------------------------------------------------------------
def blank(nb, H, B, D, seed=0):
    """A cache of noise: what no append wrote must stay."""
    rng = np.random.default_rng(seed)
    return Cache8(rng.integers(0, 256, (nb, H, B, D)).astype(np.uint8), rng.standard_normal((nb, H)).astype(np.float32))


def same(gpu, c):
    codes, steps = gpu
    assert np.array_equal(codes.cpu().numpy(), c.codes)
    assert np.array_equal(steps.cpu().numpy().view(np.uint32)[~np.isnan(c.steps)], c.steps.view(np.uint32)[~np.isnan(c.steps)])
    assert np.isnan(steps.cpu().numpy()[np.isnan(c.steps)]).all()


def grow(pa, dtype, D, H, B, chunks, seed, spread=2.0):
    """Sequences that grow by the listed chunks ([sequence] -> tokens each), appended on both sides; everything compared each time."""
    gen = torch.Generator().manual_seed(seed)
    total = [sum(c[s] for c in chunks) for s in range(len(chunks[0]))]
    tables, nb = paged(gen, total, B)
    ref = [blank(nb, H, B, D, seed + i) for i in range(2)]
    gpu = [on_gpu(c) for c in ref]
    lens = [0] * len(total)
    for fresh in chunks:
        lens = [n + c for n, c in zip(lens, fresh)]
        start = np.cumsum([0] + list(fresh))
        T = int(start[-1])
        rows = [(torch.randn(T, H, D, generator=gen) * torch.exp(spread * torch.randn(T, H, 1, generator=gen))).to(TD[dtype]) for _ in range(2)]
        pa.pa_cache_append_q8(rows[0].cuda(), rows[1].cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), gpu[0][0], gpu[1][0],
                              gpu[0][1], gpu[1][1], query_start=torch.tensor(start, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        assert pa.pa_get_device_status() == 0
        for c, x in zip(ref, rows):
            for s, n in enumerate(lens):
                c.append(tables[s].numpy(), n, x[start[s]:start[s + 1]].float().numpy())
        for g, c in zip(gpu, ref):
            same(g, c)
    return tables, lens, ref, gpu


@pytest.mark.parametrize("dtype,D", [("f16", 128), ("bf16", 128), ("f16", 64), ("bf16", 64)])
@pytest.mark.parametrize("H,B", [(1, 8), (3, 16), (8, 32), (5, 64), (2, 128), (3, 256)])
def test_bytes_follow_the_definition(pa, dtype, D, H, B):
    chunks = [[0, 1, B, 3 * B + 5, B - 1], [1, 0, 1, 7, 1], [1, 2, 2 * B, 1, 0], [B - 2, 1, 3, 0, 1], [1, 1, 1, 1, 1], [0, 0, 0, 0, 0], [17, 300, 1, 2, 40]]
    tables, lens, ref, gpu = grow(pa, dtype, D, H, B, chunks, B + H + D)
    # read back, some slots twice, padding among them
    slots = torch.cat([tables[s, torch.arange(n) // B] * B + torch.arange(n) % B for s, n in enumerate(lens)]).to(torch.int32)
    slots = torch.cat([slots, slots[:5], torch.tensor([-1], dtype=torch.int32)])
    for out_type in ("f16", "bf16"):
        out = [torch.full((len(slots), H, D), 9.0, dtype=TD[out_type], device="cuda") for _ in range(2)]
        pa.pa_cache_read_q8(gpu[0][0], gpu[1][0], gpu[0][1], gpu[1][1], slots.cuda(), out[0], out[1])
        torch.cuda.synchronize()
        assert pa.pa_get_device_status() == 0
        for c, o in zip(ref, out):
            f, at = slots[:-1].numpy() // B, slots[:-1].numpy() % B
            want = (c.codes[f, :, at].astype(np.float32) - 128) * c.steps[f][..., None]     # one rounding to fp32
            assert torch.equal(o[:-1].cpu(), torch.from_numpy(want).to(TD[out_type]))
            assert (o[-1] == 9).all()


@pytest.mark.parametrize("dtype,D,H,B", [("f16", 128, 37, 16), ("bf16", 64, 37, 8), ("bf16", 128, 9, 256), ("f16", 64, 70, 128)])
def test_steps_of_about_one_token(pa, dtype, D, H, B):
    """No more new tokens than sequences: most of them alone in their frames, some two or three, some over a frame's end, and more heads than a block takes."""
    chunks = [[1, 1, 1, 1, 1], [0, 2, 0, 1, 2], [0, 3, 1, 0, 1], [B, B, B, B, B], [1, 1, 1, 1, 1], [5, 0, 0, 0, 0], [1, 1, 1, 1, 1], [0, 0, 4, 0, 1]] + [[1, 1, 1, 1, 1]] * 10
    grow(pa, dtype, D, H, B, chunks, B + H, spread=3.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_one_token_at_a_time(pa, dtype):
    """Two frames filled token by token, in the form without query_start; an empty sequence beside them is skipped."""
    H, D, B = 2, 128, 16
    gen = torch.Generator().manual_seed(2)
    tables, nb = paged(gen, [32, 0, 20], B)
    ref = [blank(nb, H, B, D, i) for i in range(2)]
    gpu = [on_gpu(c) for c in ref]
    for n in range(1, 33):
        lens = [n, 0, min(n, 20)]
        rows = [(torch.randn(3, H, D, generator=gen) * 2.0 ** float(4 * torch.randn(1, generator=gen))).to(TD[dtype]) for _ in range(2)]
        if n > 20:
            lens[2] = 0
        pa.pa_cache_append_q8(rows[0].cuda(), rows[1].cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), gpu[0][0], gpu[1][0],
                              gpu[0][1], gpu[1][1])
        for c, x in zip(ref, rows):
            for s in (0, 2):
                if lens[s]:
                    c.append(tables[s].numpy(), lens[s], x[s:s + 1].float().numpy())
    assert pa.pa_get_device_status() == 0
    for g, c in zip(gpu, ref):
        same(g, c)


@pytest.mark.parametrize("kind", ["steps", "some", "chunks", "null"])
def test_thousands_of_sequences(pa, kind):
    """Sequences are found by a search: of single tokens, of none or a few, of chunks over several frames."""
    S, H, D, B = 3333, 1, 64, 8
    gen = torch.Generator().manual_seed(12)
    fresh = {"steps": torch.ones(S), "some": torch.randint(0, 3, (S,), generator=gen) * (torch.rand(S, generator=gen) < 0.5),
             "chunks": torch.randint(0, 20, (S,), generator=gen), "null": torch.ones(S)}[kind].int().tolist()
    lens = [int(n) + c for n, c in zip(torch.randint(0, 30, (S,), generator=gen), fresh)]
    if kind == "null":
        lens = [0 if s % 7 == 3 else n for s, n in enumerate(lens)]
        fresh = [min(n, 1) for n in lens]
    tables, nb = paged(gen, lens, B)
    c = [cache8(gen, tables, [n - f for n, f in zip(lens, fresh)], nb, H, B, D, "f16") for _ in range(2)]
    gpu = [on_gpu(x) for x in c]
    start = np.arange(S + 1) if kind == "null" else np.cumsum([0] + fresh)
    rows = [(4 * torch.randn(int(start[-1]), H, D, generator=gen)).half() for _ in range(2)]
    qs = None if kind == "null" else torch.tensor(start, dtype=torch.int32).cuda()
    pa.pa_cache_append_q8(rows[0].cuda(), rows[1].cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), gpu[0][0], gpu[1][0],
                          gpu[0][1], gpu[1][1], query_start=qs)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == 0
    for x, r, g in zip(c, rows, gpu):
        for s, n in enumerate(lens):
            x.append(tables[s].numpy(), n, r[start[s]:start[s] + fresh[s]].float().numpy())
        same(g, x)


def test_corner_frames(pa):
    """Zeros, one value, the range's ends, NaN, infinities, frames that were NaN, codes next to a border."""
    D, B, H = 64, 8, 1
    x = torch.zeros(12, 8, H, D, dtype=torch.bfloat16)                  # frames
    x[1] = 3.5
    x[2, 0, 0, :2] = torch.tensor([-1e30, 1e30])
    x[3, 4, 0, 5] = float("nan")
    x[4, 0, 0, 40] = float("-inf")
    x[5] = 1e-30
    x[6, :, 0] = torch.linspace(-127, 127, 8 * D).reshape(8, D).bfloat16()
    x[7, :, 0] = (torch.arange(8 * D).reshape(8, D) % 255 - 127 + 0.5).bfloat16()
    x[7, 0, 0, 0] = 127
    x[8] = 2.0 ** -60
    x[9] = -(2.0 ** 60)
    x[10, :, 0] = 2.0 ** -133                                           # bf16's subnormal numbers
    x[11] = 65504
    tables = torch.randperm(12, generator=torch.Generator().manual_seed(1)).to(torch.int32)[:, None]
    ref = [blank(12, H, B, D, i) for i in range(2)]
    gpu = [on_gpu(c) for c in ref]
    for n, m in ((5, 5), (7, 2), (8, 1)):                               # 5 tokens, 2 more, the last
        rows = x[:, n - m:n].reshape(12 * m, H, D)
        lens = torch.full((12,), n, dtype=torch.int32)
        start = torch.arange(13, dtype=torch.int32) * m
        other = rows.flip(-1).contiguous()
        pa.pa_cache_append_q8(rows.cuda(), other.cuda(), tables.cuda(), lens.cuda(), gpu[0][0], gpu[1][0], gpu[0][1], gpu[1][1], query_start=start.cuda())
        for c, y in zip(ref, (rows, other)):
            for s in range(12):
                c.append(tables[s].numpy(), n, y[s * m:s * m + m].float().numpy())
        for g, c in zip(gpu, ref):
            same(g, c)
    assert pa.pa_get_device_status() == 0
    assert np.isnan(ref[0].steps[int(tables[3, 0])]).all() and np.isnan(ref[0].steps[int(tables[4, 0])]).all()


def test_append_strided_rows_steps_and_tables(pa):
    H, D, B = 3, 64, 16
    gen = torch.Generator().manual_seed(5)
    lens, fresh = [40, 17, 5], [9, 17, 1]
    tables, nb = paged(gen, lens, B)
    start = np.cumsum([0] + fresh)
    T = int(start[-1])
    wide = torch.full((2, T, H * D + 16), float("nan"), dtype=torch.float16)
    wide[:, :, : H * D] = torch.randn(2, T, H * D, generator=gen).half()
    rows = wide[:, :, : H * D].reshape(2, T, H, D)
    ref = [cache8(gen, tables, [n - c for n, c in zip(lens, fresh)], nb, H, B, D, "f16") for _ in range(2)]
    gpu = [on_gpu(c) for c in ref]
    steps = torch.full((2, nb, 7), 5.0, device="cuda")
    for i in range(2):
        steps[i, :, :3] = gpu[i][1]
    t = torch.full((3, 9), 10 ** 9, dtype=torch.int32)
    t[:, : tables.shape[1]] = tables
    gw, gt = wide.cuda(), t.cuda()
    out = [gw[i, :, : H * D].unflatten(1, (H, D)) for i in range(2)]
    pa.pa_cache_append_q8(out[0], out[1], gt[:, : tables.shape[1]], torch.tensor(lens, dtype=torch.int32).cuda(), gpu[0][0], gpu[1][0],
                          steps[0, :, :3], steps[1, :, :3], query_start=torch.tensor(start, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == 0
    for i, c in enumerate(ref):
        for s, n in enumerate(lens):
            c.append(tables[s].numpy(), n, rows[i, start[s]:start[s + 1]].float().numpy())
        same((gpu[i][0], steps[i, :, :3].contiguous()), c)
    assert (steps[:, :, 3:] == 5).all()


def test_append_bad_arguments_on_the_device(pa):
    """Bad lengths, ranges and frames: their sequences are skipped, the others are written."""
    H, D, B = 2, 64, 8
    gen = torch.Generator().manual_seed(6)
    tables, nb = paged(gen, [20] * 6, B)
    ref = [cache8(gen, tables, [17] * 6, nb, H, B, D, "f16") for _ in range(2)]
    gpu = [on_gpu(c) for c in ref]
    rows = [torch.randn(18, H, D, generator=gen).half() for _ in range(2)]
    lens = torch.tensor([20, 25, 2, -1, 20, 20], dtype=torch.int32)      # 25: more than the table; 2: fewer than its rows
    start = torch.arange(7, dtype=torch.int32) * 3
    bad = tables.clone()
    bad[4, 2] = nb
    pa.pa_cache_append_q8(rows[0].cuda(), rows[1].cuda(), bad.cuda(), lens.cuda(), gpu[0][0], gpu[1][0], gpu[0][1], gpu[1][1], query_start=start.cuda())
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_LEN | pa.PA_DEV_BAD_BLOCK
    for i, c in enumerate(ref):
        for s in (0, 5):
            c.append(tables[s].numpy(), 20, rows[i][3 * s:3 * s + 3].float().numpy())
        same(gpu[i], c)
    # ranges outside the rows, and out of order
    for start in ([0, 3, 6, 9, 12, 15, 19], [0, 3, 2, 9, 12, 15, 18], [-1, 3, 6, 9, 12, 15, 18]):
        pa.pa_cache_append_q8(rows[0].cuda(), rows[1].cuda(), tables.cuda(), torch.full((6,), 20, dtype=torch.int32).cuda(), gpu[0][0], gpu[1][0],
                              gpu[0][1], gpu[1][1], query_start=torch.tensor(start, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        assert pa.pa_get_device_status() == pa.PA_DEV_BAD_LEN


def test_read_padding_and_bad_slots(pa):
    kc, vc = (torch.randint(0, 256, (2, 1, 8, 64), device="cuda").to(torch.uint8) for _ in range(2))
    ks, vs = (torch.rand(2, 1, device="cuda") for _ in range(2))
    slots = torch.tensor([-1, 16, 3, 3], dtype=torch.int32, device="cuda")
    ko, vo = (torch.full((4, 1, 64), 5.0, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pa_cache_read_q8(kc, vc, ks, vs, slots, ko, vo)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_SLOT
    assert (ko[:2] == 5).all() and (vo[:2] == 5).all()
    assert torch.equal(ko[2:], ((kc[0, :, 3].float() - 128) * ks[0]).half().expand(2, 1, 64))


def test_frames_behind_4_gib(pa):
    """Appends, reads and attention in frames whose offsets pass 32 bits."""
    H, D, B, nb = 8, 128, 16, 300_000                                   # 4.9 GB a cache
    gen = torch.Generator().manual_seed(7)
    caches = [torch.zeros(nb, H, B, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    steps = [torch.zeros(nb, H, device="cuda") for _ in range(2)]
    tables = torch.tensor([[nb - 1, nb - 5, 0]], dtype=torch.int32)
    rows = [torch.randn(40, H, D, generator=gen).half() for _ in range(2)]
    n = torch.tensor([40], dtype=torch.int32).cuda()
    pa.pa_cache_append_q8(rows[0].cuda(), rows[1].cuda(), tables.cuda(), n, caches[0], caches[1], steps[0], steps[1],
                          query_start=torch.tensor([0, 40], dtype=torch.int32).cuda())
    ref = [blank(3, H, B, D) for _ in range(2)]
    for c, x, g, st in zip(ref, rows, caches, steps):
        c.append([0, 1, 2], 40, x.float().numpy())
        assert np.array_equal(g[tables[0].long().cuda()].cpu().numpy()[:2], c.codes[:2])
        assert np.array_equal(st[tables[0].long().cuda()].cpu().numpy(), c.steps)
    q = torch.randn(1, 4 * H, D, generator=gen).half()
    out = torch.empty_like(q, device="cuda")
    pa.pa_decode_q8(q.cuda(), caches[0], caches[1], steps[0], steps[1], tables.cuda(), n, 0.1, out)
    k, v = (c.values([0, 1, 2], 40) for c in ref)
    want = attend_seen(host64(q[0]), k, v, 39, 0, 0, 0.1)
    assert (np.abs(host64(out[0]) - want) <= attention_tolerance(want, torch.float16, host64(q[0]), k, v, 0.1, 2.0 ** -22)).all()
    slots = torch.tensor([(nb - 1) * B + 3, 5], dtype=torch.int32).cuda()
    ko, vo = (torch.empty(2, H, D, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pa_cache_read_q8(caches[0], caches[1], steps[0], steps[1], slots, ko, vo)
    assert torch.equal(ko[0].cpu(), torch.from_numpy(k[3].astype(np.float32)).half())
    assert torch.equal(vo[1].cpu(), torch.from_numpy(v[37].astype(np.float32)).half())
    assert pa.pa_get_device_status() == 0


# ---- decode --------------------------------------------------------------------------------------------
def decode_case(lens, H, g, D, B, dtype, seed, window=0, sinks=0, q_scale=1.0, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    tables, nb = window_tables(gen, lens, [1] * len(lens), B, window, sinks)
    kc, vc = (cache8(gen, tables, lens, nb, H, B, D, dtype, spread) for _ in range(2))
    q = (torch.randn(len(lens), H * g, D, generator=gen) * q_scale).to(TD[dtype])
    return q, kc, vc, torch.where(tables < 0, 10 ** 9, tables), torch.tensor(lens, dtype=torch.int32)


def reference(case, window, sinks, scale, s):
    q, kc, vc, tables, lens = case
    n, B = int(lens[s]), kc.codes.shape[2]
    j = seen(n - 1, window, sinks)
    f = tables[s].numpy()[j // B]
    k, v = ((c.codes[f, :, j % B].astype(np.float64) - 128) * c.steps[f].astype(np.float64)[..., None] for c in (kc, vc))
    return attend_seen(host64(q[s]), k, v, len(k) - 1, 0, 0, scale), k, v


def check_decode(pa, case, scale, dtype, window=0, sinks=0, seqs=None):
    q, kc, vc, tables, lens = case
    (k, ks), (v, vs) = on_gpu(kc), on_gpu(vc)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    pa.pa_decode_q8(q.cuda(), k, v, ks, vs, tables.cuda(), lens.cuda(), scale, out, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == 0
    got = host64(out)
    for s in range(len(lens)) if seqs is None else seqs:
        ref, kk, vv = reference(case, window, sinks, scale, s)
        tol = attention_tolerance(ref, TD[dtype], host64(q[s]), kk, vv, scale, 2.0 ** -22)
        err = np.abs(got[s] - ref)
        assert (err <= tol).all(), (s, int(lens[s]), float((err - tol).max()), float(err.max()))
    return out


LENS = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 64, 100, 255, 257, 700]


@pytest.mark.parametrize("B", [8, 16, 32, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,g", [(1, 1), (3, 4), (2, 7), (1, 13), (2, 16)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_lengths(pa, B, D, H, g, dtype):
    check_decode(pa, decode_case(LENS, H, g, D, B, dtype, B + D + H + g), D ** -0.5, dtype)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (7, 1), (16, 16), (33, 17), (100, 4), (256, 100), (10000, 3)])
@pytest.mark.parametrize("dtype,D,H,g,B", [("f16", 128, 2, 4, 16), ("bf16", 64, 3, 1, 8), ("bf16", 128, 1, 7, 256), ("f16", 64, 1, 16, 32)])
def test_decode_windows(pa, dtype, D, H, g, B, window, sinks):
    check_decode(pa, decode_case(LENS, H, g, D, B, dtype, B + window, window, sinks), D ** -0.5, dtype, window, sinks)


@pytest.mark.parametrize("g", [1, 4, 8])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_split_contexts(pa, g, dtype):
    check_decode(pa, decode_case([20000, 3, 0, 5000, 1], 1, g, 128, 16, dtype, 3), 128 ** -0.5, dtype)


def test_decode_many_sequences(pa):
    lens = [(i * 7) % 50 for i in range(1000)]
    check_decode(pa, decode_case(lens, 4, 2, 64, 16, "bf16", 4), 0.125, "bf16", seqs=range(0, 1000, 37))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("q_scale", [12.0, 1e-3, 0.0])
def test_decode_value_ranges(pa, dtype, q_scale):
    check_decode(pa, decode_case([500, 17, 64], 2, 4, 128, 16, dtype, 6, q_scale=q_scale), 128 ** -0.5, dtype)


def test_decode_steps_far_apart(pa):
    """Frames whose values are 2^20 times others': sums in units of the largest step so far, which moves up and stays."""
    for order in (1, -1):
        gen = torch.Generator().manual_seed(8)
        q, kc, vc, tables, lens = decode_case([640, 100], 1, 4, 64, 16, "bf16", 8)
        for j in range(40):
            f = int(tables[0, j])
            x = (torch.randn(16, 1, 64, generator=gen) * 2.0 ** (order * (j - 20))).bfloat16().float().numpy()
            vc.append([f], 16, x)
        check_decode(pa, (q, kc, vc, tables, lens), 0.1, "bf16")


def test_decode_tiny_and_huge_values(pa):
    for size in (2.0 ** -50, 2.0 ** 50):
        gen = torch.Generator().manual_seed(9)
        q, kc, vc, tables, lens = decode_case([100], 1, 1, 64, 16, "bf16", 9)
        for j in range(7):
            n = min(16, 100 - 16 * j)
            for c, x in ((vc, size), (kc, 1 / size)):
                c.append([int(tables[0, j])], n, (torch.randn(n, 1, 64, generator=gen) * x).bfloat16().float().numpy())
        q = (q.float() * size).bfloat16()
        check_decode(pa, (q, kc, vc, tables, lens), 0.1, "bf16")


def test_decode_queries_beyond_fp16(pa):
    for q_scale, scale in ((1e6, 1e-7), (1e-9, 1e8)):
        check_decode(pa, decode_case([300, 40], 2, 2, 64, 16, "bf16", 8, q_scale=q_scale), scale, "bf16")


def test_decode_nan_frames_show(pa):
    """A frame with a NaN step makes its sequence's rows of that head NaN, and no others; a window that leaves it out does not."""
    q, kc, vc, tables, lens = decode_case([100, 60], 2, 2, 64, 16, "f16", 11)
    kc.steps[int(tables[0, 1]), 1] = np.nan
    vc.steps[int(tables[1, 0]), 0] = np.nan
    (k, ks), (v, vs) = on_gpu(kc), on_gpu(vc)
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    pa.pa_decode_q8(q.cuda(), k, v, ks, vs, tables.cuda(), lens.cuda(), 0.1, out)
    nan = torch.isnan(out).all(-1).cpu()
    assert nan.tolist() == [[False, False, True, True], [True, True, False, False]]
    assert torch.isfinite(out[~nan.cuda()]).all()
    pa.pa_decode_q8(q.cuda(), k, v, ks, vs, tables.cuda(), lens.cuda(), 0.1, out, window=40, sinks=0)
    assert torch.isfinite(out).all()
    assert pa.pa_get_device_status() == 0


def test_decode_bad_indexes(pa):
    q, kc, vc, tables, lens = decode_case([100, 50, 40, 30], 2, 4, 64, 16, "f16", 10)
    check_decode(pa, (q, kc, vc, tables, lens), 0.125, "f16")
    (k, ks), (v, vs) = on_gpu(kc), on_gpu(vc)
    bad_t, bad_l = tables.clone(), lens.clone()
    bad_t[0, 3] = kc.codes.shape[0]
    bad_t[1, 0] = -5
    bad_l[2] = tables.shape[1] * 16 + 1
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    pa.pa_decode_q8(q.cuda(), k, v, ks, vs, bad_t.cuda(), bad_l.cuda(), 0.125, out)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_BLOCK | pa.PA_DEV_BAD_LEN
    assert not out[:3].any()
    ref, kk, vv = reference((q, kc, vc, tables, lens), 0, 0, 0.125, 3)
    assert (np.abs(host64(out[3]) - ref) <= attention_tolerance(ref, torch.float16, host64(q[3]), kk, vv, 0.125, 2.0 ** -22)).all()
    check_decode(pa, (q, kc, vc, tables, lens), 0.125, "f16")


def test_decode_and_read_strided_rows_steps_and_tables(pa):
    case = decode_case([100, 50, 40], 3, 2, 64, 16, "f16", 16)
    ref = check_decode(pa, case, 0.1, "f16")
    q, kc, vc, tables, lens = case
    (k, ks), (v, vs) = on_gpu(kc), on_gpu(vc)
    nb = k.shape[0]
    steps = torch.full((2, nb, 9), float("nan"), device="cuda")
    steps[0, :, 1:4], steps[1, :, 1:4] = ks, vs
    wide_q = torch.full((3, 6 * 64 + 8), float("nan"), dtype=torch.float16, device="cuda")
    wide_q[:, : 6 * 64] = q.flatten(1).cuda()
    wide_o = torch.full((3, 6 * 64 + 16), 9.0, dtype=torch.float16, device="cuda")
    wide_t = torch.full((3, 40), -7, dtype=torch.int32, device="cuda")
    wide_t[:, : tables.shape[1]] = tables.cuda()
    pa.pa_decode_q8(wide_q[:, : 6 * 64].unflatten(1, (6, 64)), k, v, steps[0, :, 1:4], steps[1, :, 1:4], wide_t[:, : tables.shape[1]], lens.cuda(), 0.1,
                    wide_o[:, : 6 * 64].unflatten(1, (6, 64)))
    assert torch.equal(wide_o[:, : 6 * 64].unflatten(1, (6, 64)), ref)
    assert (wide_o[:, 6 * 64:] == 9).all()
    slots = torch.arange(nb * 16, dtype=torch.int32).cuda()
    a, b = (torch.full((2, nb * 16, 3, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wide = torch.full((2, nb * 16, 3 * 64 + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    pa.pa_cache_read_q8(k, v, ks, vs, slots, a[0], a[1])
    out = wide[:, :, : 3 * 64].unflatten(2, (3, 64))
    pa.pa_cache_read_q8(k, v, steps[0, :, 1:4], steps[1, :, 1:4], slots, out[0], out[1])
    assert torch.equal(out.nan_to_num(5), a.nan_to_num(5)) and (wide[:, :, 3 * 64:] == 9).all()
    assert pa.pa_get_device_status() == 0


def test_decode_same_bits_every_time(pa):
    q, kc, vc, tables, lens = decode_case([9000, 40, 777, 2048], 2, 4, 128, 32, "bf16", 15)
    (k, ks), (v, vs) = on_gpu(kc), on_gpu(vc)
    q, tables, lens = q.cuda(), tables.cuda(), lens.cuda()
    first = torch.empty_like(q)
    pa.pa_decode_q8(q, k, v, ks, vs, tables, lens, 0.1, first)
    for _ in range(20):
        again = torch.empty_like(q)
        pa.pa_decode_q8(q, k, v, ks, vs, tables, lens, 0.1, again)
        assert torch.equal(first, again)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [3, 5, 8, 12, 16])
def test_decode_joins_of_many_queries(pa, g, D):
    """A head of 20000 tokens is joined in groups; of 400 heads of 300 tokens most are in pieces, and a block joins several."""
    check_decode(pa, decode_case([20000, 3, 0, 5000, 1], 1, g, D, 16, "f16", 30 + g), D ** -0.5, "f16")
    check_decode(pa, decode_case([300 - i % 7 for i in range(200)], 2, g, D, 16, "bf16", 31 + g), D ** -0.5, "bf16", seqs=range(0, 200, 3))
