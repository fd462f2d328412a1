"""The 4-bit cache: its bytes, its values read back, and decode attention over it."""

import numpy as np
import pytest
import torch

from oracle.operators import attend, cos_sin_table, quantise_q4, rotate, values_q4
from tests._operators_common import TD, attention_tolerance, half_step, host64, paged

pytestmark = pytest.mark.gpu


def rows(gen, *shape, dtype):
    centre = torch.randn(shape[-1], generator=gen) * (torch.rand(shape[-1], generator=gen) < 0.1)
    return (torch.randn(*shape, generator=gen) + 3 * centre).to(TD[dtype])


# ---- append and read -----------------------------------------------------------------------------------
@pytest.mark.parametrize("mode", ["plain", "half", "interleaved"])
@pytest.mark.parametrize("dtype,D,R", [("f16", 128, 128), ("bf16", 128, 48), ("f16", 64, 64), ("bf16", 64, 16)])
@pytest.mark.parametrize("T,H,Hq,B", [(1, 1, 1, 16), (5, 3, 6, 8), (130, 2, 2, 64), (333, 8, 3, 256)])
def test_bytes_follow_the_definition(pa, mode, dtype, D, R, T, H, Hq, B):
    g = torch.Generator().manual_seed(T + D)
    k, v, q = rows(g, T, H, D, dtype=dtype), rows(g, T, H, D, dtype=dtype), rows(g, T, Hq, D, dtype=dtype)
    nb = -(-T // B) + 1
    slots = torch.randperm(nb * B, generator=g)[:T].to(torch.int32)
    pos = torch.randint(0, 300, (T,), generator=g, dtype=torch.int32)
    table = cos_sin_table(300, R)
    kc, vc = (torch.full((nb, H, B, 5 * D // 8), 77, dtype=torch.uint8, device="cuda") for _ in range(2))
    qo = torch.empty_like(q, device="cuda")
    more = {} if mode == "plain" else dict(positions=pos.cuda(), cos_sin=torch.from_numpy(table).cuda(), q=q.cuda(), q_out=qo,
                                           interleaved=mode == "interleaved")
    pa.pa_cache_append_q4(k.cuda(), v.cuda(), slots.cuda(), kc, vc, **more)
    ko, vo = (torch.empty(T, H, D, dtype=TD[dtype], device="cuda") for _ in range(2))
    pa.pa_cache_read_q4(kc, vc, slots.cuda(), ko, vo)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == 0
    turned = k.float().numpy()
    if mode != "plain":
        turned = rotate(turned, table, pos.numpy(), mode == "interleaved")
        ref = rotate(host64(q), table, pos.numpy(), mode == "interleaved")
        assert (np.abs(host64(qo) - ref) <= half_step(TD[dtype]) * np.abs(ref) + 3 * 2.0 ** -24 * 2 * np.abs(host64(q)).max()).all()
    for cache, x, got in ((kc, turned, ko), (vc, v.float().numpy(), vo)):
        want = quantise_q4(x)
        flat = cache.transpose(1, 2).flatten(0, 1).cpu()
        assert np.array_equal(flat[slots.long()].numpy(), want)
        rest = torch.ones(nb * B, dtype=torch.bool)
        rest[slots.long()] = False
        assert (flat[rest] == 77).all()
        assert torch.equal(got.cpu(), torch.from_numpy(values_q4(want)).to(TD[dtype]))


def test_corner_groups(pa):
    """Groups of one value, tiny and huge ranges, values beyond fp16, NaN and infinities."""
    D, B = 64, 8
    x = torch.zeros(8, 1, D, dtype=torch.bfloat16)
    x[1] = 3.5
    x[2, 0, :2] = torch.tensor([-1e30, 1e30])
    x[3, 0, 5] = float("nan")
    x[4, 0, 40] = float("-inf")
    x[5] = torch.linspace(1e-7, 9e-7, D)
    x[6] = 1000 + torch.linspace(0, 4, D)
    x[7, 0] = torch.linspace(-60000, 60000, D)
    slots = torch.arange(8, dtype=torch.int32).cuda()
    kc, vc = (torch.zeros(1, 1, B, 40, dtype=torch.uint8, device="cuda") for _ in range(2))
    pa.pa_cache_append_q4(x.cuda(), x.flip(0).contiguous().cuda(), slots, kc, vc)
    ko, vo = (torch.empty(8, 1, D, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pa_cache_read_q4(kc, vc, slots, ko, vo)
    want = quantise_q4(x.float().numpy())
    assert np.array_equal(kc[0, 0].cpu().numpy(), want[:, 0])
    assert np.array_equal(vc[0, 0].cpu().numpy(), want[::-1, 0])
    assert np.array_equal(host64(ko), values_q4(want), equal_nan=True)
    assert np.array_equal(host64(vo), values_q4(want[::-1]), equal_nan=True)
    assert torch.isnan(ko[3, 0, :32]).all() and torch.isfinite(ko[3, 0, 32:]).all() and torch.isnan(ko[4, 0, 32:]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_borders_between_codes(pa, dtype):
    """Elements on a border between two codes and next to it, and ranges far below their offset's rounding: each code
    is that of the division."""
    g = torch.Generator().manual_seed(41)
    n, D, B = 4096, 128, 16
    step = (torch.rand(n, 1, generator=g) + 0.5) * 2.0 ** torch.randint(-22, 11, (n, 1), generator=g)
    step = step.half().float()
    border = torch.randint(0, 31, (n, D), generator=g).float() * 0.5
    border[:, 0::32], border[:, 1::32] = 0.0, 15.0  # the range is 15 steps
    x = (step * border).to(TD[dtype])
    near = x.view(torch.int16) + torch.randint(-1, 2, (n, D), generator=g).to(torch.int16)
    near[:, 0::32], near[:, 1::32] = x.view(torch.int16)[:, 0::32], x.view(torch.int16)[:, 1::32]
    x[n // 2:] = near.clamp(min=0).view(TD[dtype])[n // 2:]
    x = x - (torch.randint(0, 3, (n, 1), generator=g) * 7.0 * step).to(TD[dtype])
    far = (torch.randn(n, D, generator=g) * 0.02 + 1000 * torch.randn(n, 1, generator=g)).to(TD[dtype])
    x, far = (t.reshape(n // 2, 2, D) for t in (x, far))
    slots = torch.arange(n // 2, dtype=torch.int32).cuda()
    kc, vc = (torch.zeros(n // 2 // B, 2, B, 5 * D // 8, dtype=torch.uint8, device="cuda") for _ in range(2))
    pa.pa_cache_append_q4(x.cuda(), far.cuda(), slots, kc, vc)
    for cache, rows_ in ((kc, x), (vc, far)):
        got = cache.transpose(1, 2).flatten(0, 1).cpu().numpy()
        assert np.array_equal(got, quantise_q4(rows_.float().numpy()))


def test_read_padding_and_bad_slots(pa):
    kc, vc = (torch.randint(0, 200, (2, 1, 8, 40), device="cuda").to(torch.uint8) for _ in range(2))
    slots = torch.tensor([-1, 16, 3, 3], dtype=torch.int32, device="cuda")
    ko, vo = (torch.full((4, 1, 64), 5.0, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pa_cache_read_q4(kc, vc, slots, ko, vo)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_SLOT
    assert (ko[:2] == 5).all() and (vo[:2] == 5).all()
    want = values_q4(kc[0, :, 3].cpu().numpy())
    for i in (2, 3):
        assert np.array_equal(host64(ko[i]), want, equal_nan=True)


def test_copied_frames(pa):
    kc, vc = (torch.randint(0, 256, (5, 3, 16, 80), device="cuda").to(torch.uint8) for _ in range(2))
    before = kc.clone(), vc.clone()
    pa.pa_copy_blocks(kc, vc, torch.tensor([[1, 4], [0, 2]], dtype=torch.int32, device="cuda"))
    for now, was in zip((kc, vc), before):
        assert torch.equal(now[[4, 2]], was[[1, 0]]) and torch.equal(now[[0, 1, 3]], was[[0, 1, 3]])


# ---- decode --------------------------------------------------------------------------------------------
def decode_case(lens, H, g, D, B, dtype, seed, poison=True, q_scale=1.0, width=None):
    gen = torch.Generator().manual_seed(seed)
    tables, nb = paged(gen, lens, B, width=width)
    caches = []
    for _ in range(2):
        c = torch.from_numpy(quantise_q4(rows(gen, nb, H, B, D, dtype="f16").float().numpy()))
        caches.append(c)
    if poison:  # slots that hold no token: every bit set (NaN steps and offsets)
        live = torch.zeros(nb, B, dtype=torch.bool)
        for s, n in enumerate(lens):
            for j in range(-(-n // B)):
                live[tables[s, j], : n - j * B] = True
        for c in caches:
            c.transpose(1, 2)[~live] = 255
    q = (torch.randn(len(lens), H * g, D, generator=gen) * q_scale).to(TD[dtype])
    return q, caches[0], caches[1], tables, torch.tensor(lens, dtype=torch.int32)


def decode_reference(q, kc, vc, tables, lens, B, scale, s):
    """With bf16 queries a key enters its score as step * n + offset, not rounded to fp16."""
    n = int(lens[s])
    f = tables[s, : -(-n // B)].long()
    k, v = (values_q4(c[f].numpy(), rounded=c is vc or q.dtype == torch.float16).transpose(0, 2, 1, 3)
            .reshape(-1, c.shape[1], c.shape[3] // 5 * 8)[:n] for c in (kc, vc))
    return attend(host64(q[s]), k, v, scale), k, v


def check_decode(pa, case, B, scale, dtype, g, seqs=None):
    q, kc, vc, tables, lens = case
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    pa.pa_decode_q4(q.cuda(), kc.cuda(), vc.cuda(), tables.cuda(), lens.cuda(), scale, out)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == 0
    got = host64(out)
    step = 2.0 ** -22 if dtype == "f16" or g <= 4 else 2.0 ** -11   # two parts of fp16, or one
    for s in range(len(lens)) if seqs is None else seqs:
        ref, k, v = decode_reference(q, kc, vc, tables, lens, B, scale, s)
        tol = attention_tolerance(ref, TD[dtype], host64(q[s]), k, v, scale, step)
        err = np.abs(got[s] - ref)
        assert (err <= tol).all(), (s, int(lens[s]), float((err - tol).max()), float(err.max()))
    return out


@pytest.mark.parametrize("B", [8, 16, 32, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,g", [(1, 1), (3, 4), (2, 7), (2, 8), (1, 13), (2, 16), (5, 2)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_lengths(pa, B, D, H, g, dtype):
    lens = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 64, 100, 255, 257, 700]
    check_decode(pa, decode_case(lens, H, g, D, B, dtype, B + D + H + g), B, D ** -0.5, dtype, g)


@pytest.mark.parametrize("g", [1, 4, 8])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_split_contexts(pa, g, dtype):
    """Few heads and long contexts: pieces of a context joined, short ones beside it."""
    check_decode(pa, decode_case([20000, 3, 0, 5000, 1], 1, g, 128, 16, dtype, 3), 16, 128 ** -0.5, dtype, g)


def test_decode_many_sequences(pa):
    """More (sequence, head) pairs than warps on the GPU, empty ones among them."""
    lens = [(i * 7) % 50 for i in range(1000)]
    check_decode(pa, decode_case(lens, 4, 2, 64, 16, "bf16", 4), 16, 0.125, "bf16", 2, seqs=range(0, 1000, 37))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("q_scale", [12.0, 1e-3, 0.0])
def test_decode_value_ranges(pa, dtype, q_scale):
    """Sharp and flat softmax; an all-zero query attends evenly."""
    case = decode_case([500, 17, 64], 2, 4, 128, 16, dtype, 6, q_scale=q_scale)
    check_decode(pa, case, 16, 128 ** -0.5, dtype, 4)


def test_decode_queries_beyond_fp16(pa):
    """bf16 queries far outside fp16's range, brought back by the scale."""
    for q_scale, scale in ((1e6, 1e-7), (1e-9, 1e8)):
        case = decode_case([300, 40], 2, 2, 64, 16, "bf16", 8, q_scale=q_scale)
        check_decode(pa, case, 16, scale, "bf16", 2)


def test_decode_rows_in_descending_scores(pa):
    """Each key scores higher or lower than the one before, by far: the running maximum moves at every tile."""
    lens, H, D, B = [640], 1, 128, 16
    for sign in (1, -1):
        q, kc, vc, tables, n = decode_case(lens, H, 1, D, B, "f16", 9)
        k = torch.zeros(640, 1, D)
        k[:, 0, 0] = sign * torch.arange(640) * 0.5
        rowsk = torch.from_numpy(quantise_q4(k.numpy()))
        for j in range(40):
            kc[tables[0, j]] = rowsk[16 * j:16 * j + 16].transpose(0, 1)
        q.zero_()
        q[0, 0, 0] = 8.0
        check_decode(pa, (q, kc, vc, tables, n), B, 0.5, "f16", 1)


def test_decode_bad_indexes(pa):
    q, kc, vc, tables, lens = decode_case([100, 50, 40, 30], 2, 4, 64, 16, "f16", 10)
    good = check_decode(pa, (q, kc, vc, tables, lens), 16, 0.125, "f16", 4)
    bad_t, bad_l = tables.clone(), lens.clone()
    bad_t[0, 3] = kc.shape[0]
    bad_t[1, 0] = -5
    bad_l[2] = tables.shape[1] * 16 + 1
    out = torch.full_like(good, float("nan"))
    pa.pa_decode_q4(q.cuda(), kc.cuda(), vc.cuda(), bad_t.cuda(), bad_l.cuda(), 0.125, out)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_BLOCK | pa.PA_DEV_BAD_LEN
    assert not out[:3].any()
    # cut among the warps by its lengths, a batch with one of them bad sums in another order: held to the 64-bit result
    ref, k, v = decode_reference(q, kc, vc, tables, lens, 16, 0.125, 3)
    assert (np.abs(host64(out[3]) - ref) <= attention_tolerance(ref, torch.float16, host64(q[3]), k, v, 0.125, 2.0 ** -22)).all()
    bad_l[2] = -1
    pa.pa_decode_q4(q.cuda(), kc.cuda(), vc.cuda(), tables.cuda(), bad_l.cuda(), 0.125, out)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_LEN
    assert not out[2].any()
    check_decode(pa, (q, kc, vc, tables, lens), 16, 0.125, "f16", 4)   # later calls start clean


def test_decode_strided_rows_and_tables(pa):
    q, kc, vc, tables, lens = decode_case([100, 50, 40], 2, 4, 128, 16, "bf16", 12)
    ref = check_decode(pa, (q, kc, vc, tables, lens), 16, 0.1, "bf16", 4)
    wide_q = torch.full((3, 8 * 128 + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_q[:, : 8 * 128] = q.flatten(1).cuda()
    wide_o = torch.full((3, 8 * 128 + 32), 9.0, dtype=torch.bfloat16, device="cuda")
    wide_t = torch.full((3, 40), -7, dtype=torch.int32, device="cuda")
    wide_t[:, : tables.shape[1]] = tables.cuda()
    pa.pa_decode_q4(wide_q[:, : 8 * 128].view(3, 8, 128), kc.cuda(), vc.cuda(), wide_t[:, : tables.shape[1]], lens.cuda(), 0.1,
                    wide_o[:, : 8 * 128].view(3, 8, 128))
    assert torch.equal(wide_o[:, : 8 * 128].reshape(3, 8, 128), ref)
    assert (wide_o[:, 8 * 128:] == 9).all()


def test_decode_frames_behind_4_gib(pa):
    H, D, B = 8, 128, 16
    nb = 450_000                                           # 4.6 GB a cache
    q, kc, vc, tables, lens = decode_case([70, 33], H, 4, D, B, "f16", 13)
    big = [torch.empty(nb, H, B, 80, dtype=torch.uint8, device="cuda") for _ in range(2)]
    n = kc.shape[0]
    for b, c in zip(big, (kc, vc)):
        b[nb - n:] = c.cuda()
    far = torch.where(tables >= 0, tables + (nb - n), tables)
    out, ref = (torch.empty(q.shape, dtype=q.dtype, device="cuda") for _ in range(2))
    pa.pa_decode_q4(q.cuda(), big[0], big[1], far.cuda(), lens.cuda(), 0.1, out)
    pa.pa_decode_q4(q.cuda(), kc.cuda(), vc.cuda(), tables.cuda(), lens.cuda(), 0.1, ref)
    assert torch.equal(out, ref)
    assert pa.pa_get_device_status() == 0


def test_decode_empty_batches(pa):
    q, kc, vc, tables, lens = decode_case([0, 0, 0], 2, 1, 64, 16, "f16", 14)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    pa.pa_decode_q4(q.cuda(), kc.cuda(), vc.cuda(), tables.cuda(), lens.cuda(), 0.1, out)
    assert not out.any()
    none = torch.empty(3, 0, dtype=torch.int32, device="cuda")        # tables without a column
    out.fill_(float("nan"))
    pa.pa_decode_q4(q.cuda(), kc.cuda(), vc.cuda(), none, lens.cuda(), 0.1, out)
    assert not out.any()
    n = pa.pa_launch_count()
    pa.pa_decode_q4(q[:0].cuda(), kc.cuda(), vc.cuda(), tables[:0].cuda(), lens[:0].cuda(), 0.1, out[:0])
    assert pa.pa_launch_count() == n
    assert pa.pa_get_device_status() == 0


def test_decode_same_bits_every_time(pa):
    q, kc, vc, tables, lens = (x.cuda() for x in decode_case([9000, 40, 777, 2048], 2, 4, 128, 32, "bf16", 15))
    first = torch.empty_like(q)
    pa.pa_decode_q4(q, kc, vc, tables, lens, 0.1, first)
    for _ in range(20):
        again = torch.empty_like(q)
        pa.pa_decode_q4(q, kc, vc, tables, lens, 0.1, again)
        assert torch.equal(first, again)
