"""pa_cache_append_rope against the 64-bit rotation, and the writes it must not make."""

import numpy as np
import pytest
import torch

from oracle.operators import cos_sin_table, rotate
from tests._operators_common import TD, half_step, host64, tiny

pytestmark = pytest.mark.gpu


def inputs(T, H, Hq, D, B, R, dtype, seed, max_pos=500):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g).to(TD[dtype]).cuda()
    nb = -(-T // B) + 2
    d = {"k": rn(T, H, D), "v": rn(T, H, D), "q": rn(T, Hq, D) if Hq else None, "kc": rn(nb, B, H, D), "vc": rn(nb, B, H, D),
         "slots": torch.randperm(nb * B, generator=g)[:T].to(torch.int32).cuda(),
         "pos": torch.randint(0, max_pos, (T,), generator=g, dtype=torch.int32).cuda(),
         "cs": torch.from_numpy(cos_sin_table(max_pos, R)).cuda()}
    return d


def close(got, x, table, pos, inter, dtype):
    """Within half a step of the type, and three roundings to fp32 of numbers below |x1| + |x2|."""
    ref = rotate(x, table, pos, inter)
    size = rotate(np.abs(x), np.abs(table), pos, inter)
    R = table.shape[1]
    a, b = (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))
    top = np.abs(x[..., a]) + np.abs(x[..., b])
    size[..., a] = top
    size[..., b] = top
    exact = np.ones(x.shape[-1], bool)
    exact[:R] = False
    err = np.abs(got - ref)
    assert (err <= half_step(TD[dtype]) * np.abs(ref) + 3 * 2.0 ** -24 * size + tiny(TD[dtype])).all(), err.max()
    assert not err[..., exact].any()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,D,R", [("f16", 128, 128), ("bf16", 128, 64), ("f16", 64, 16), ("f32", 128, 96), ("f32", 64, 64),
                                       ("bf16", 80, 32), ("f16", 256, 256), ("f16", 96, 80), ("f32", 16, 16)])
@pytest.mark.parametrize("T,H,Hq", [(1, 1, 0), (3, 2, 8), (70, 5, 5), (700, 3, 1)])
def test_rotates_and_appends(pa, dtype, D, R, inter, T, H, Hq):
    d = inputs(T, H, Hq, D, 16, R, dtype, T + D + R)
    kc0, vc0 = d["kc"].clone(), d["vc"].clone()
    q_out = None if not Hq else torch.full_like(d["q"], float("nan"))
    pa.pa_cache_append_rope(d["k"], d["v"], d["slots"], d["kc"], d["vc"], d["pos"], d["cs"], q=d["q"], q_out=q_out,
                            interleaved=inter)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == 0
    slots, pos, table = d["slots"].long(), d["pos"].cpu().numpy(), d["cs"].double().cpu().numpy()
    close(host64(d["kc"].flatten(0, 1)[slots]), host64(d["k"]), table, pos, inter, dtype)
    assert torch.equal(d["vc"].flatten(0, 1)[slots], d["v"])
    if Hq:
        close(host64(q_out), host64(d["q"]), table, pos, inter, dtype)
    rest = torch.ones(kc0.shape[0] * 16, dtype=torch.bool, device="cuda")
    rest[slots] = False
    for now, before in ((d["kc"], kc0), (d["vc"], vc0)):
        assert torch.equal(now.flatten(0, 1)[rest], before.flatten(0, 1)[rest])


@pytest.mark.parametrize("inter", [False, True])
def test_queries_in_place_and_strided_rows(pa, inter):
    """q_out = q; keys, values and queries as slices of one projection's output."""
    T, H, Hq, D = 37, 4, 12, 128
    d = inputs(T, H, Hq, D, 8, 128, "bf16", 5)
    wide = torch.cat([d["q"].flatten(1), d["k"].flatten(1), d["v"].flatten(1)], dim=1)
    q = wide[:, : Hq * D].view(T, Hq, D)
    k = wide[:, Hq * D:(Hq + H) * D].view(T, H, D)
    v = wide[:, (Hq + H) * D:].view(T, H, D)
    cs = torch.zeros(500, 132, device="cuda")[:, :128]
    cs.copy_(d["cs"])
    pa.pa_cache_append_rope(k, v, d["slots"], d["kc"], d["vc"], d["pos"], cs, q=q, q_out=q, interleaved=inter)
    torch.cuda.synchronize()
    pos, table = d["pos"].cpu().numpy(), d["cs"].double().cpu().numpy()
    close(host64(q), host64(d["q"]), table, pos, inter, "bf16")
    close(host64(d["kc"].flatten(0, 1)[d["slots"].long()]), host64(d["k"]), table, pos, inter, "bf16")
    assert torch.equal(d["vc"].flatten(0, 1)[d["slots"].long()], d["v"])
    assert torch.equal(k, d["k"]) and torch.equal(v, d["v"])


@pytest.mark.parametrize("q4", [False, True])
def test_padding_and_bad_indexes(pa, q4):
    T, H, Hq, D, B = 6, 2, 4, 64, 16
    d = inputs(T, H, Hq, D, B, 64, "f16", 9)
    kc, vc = (d["kc"], d["vc"]) if not q4 else (torch.zeros(4, H, B, 40, dtype=torch.uint8, device="cuda") for _ in range(2))
    nslots = kc.shape[0] * B
    #          live, padded slot, padded position, slot behind the cache, position behind the table, live
    slots = [3, -1, 5, nslots, 7, 0]
    pos = [4, 5, -1, 6, 500, 499]
    d["slots"].copy_(torch.tensor(slots, dtype=torch.int32))
    d["pos"].copy_(torch.tensor(pos, dtype=torch.int32))
    out = torch.full_like(d["q"], 7.0)
    before = [kc.clone(), vc.clone()]
    call = pa.pa_cache_append_q4 if q4 else pa.pa_cache_append_rope
    call(d["k"], d["v"], d["slots"], kc, vc, d["pos"], d["cs"], q=d["q"], q_out=out)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == pa.PA_DEV_BAD_SLOT | pa.PA_DEV_BAD_POS
    assert pa.pa_get_device_status() == 0
    table = d["cs"].double().cpu().numpy()
    live = [0, 1, 3, 5]
    close(host64(out[live]), host64(d["q"][live]), table, np.array(pos)[live], False, "f16")
    assert (out[[2, 4]] == 7.0).all()
    written = torch.zeros(nslots, dtype=torch.bool, device="cuda")
    written[[3, 0]] = True
    for now, was in zip((kc, vc), before):
        if q4:
            now, was = now.transpose(1, 2), was.transpose(1, 2)
        same = (now == was).flatten(0, 1).flatten(1).all(1)
        assert torch.equal(same, ~written)


def test_frames_behind_4_gib(pa):
    """Byte offsets that pass 32 bits."""
    H, D, B = 8, 128, 16
    nb = 140_000                                           # 4.6 GB a cache
    kc, vc = (torch.empty(nb, B, H, D, dtype=torch.float16, device="cuda") for _ in range(2))
    d = inputs(2, H, 0, D, B, 128, "f16", 11)
    slots = torch.tensor([nb * B - 1, 2 ** 17 * B + 5], dtype=torch.int32, device="cuda")
    kc.view(-1, H, D)[slots.long()] = 0
    pa.pa_cache_append_rope(d["k"], d["v"], slots, kc, vc, d["pos"], d["cs"])
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == 0
    close(host64(kc.view(-1, H, D)[slots.long()]), host64(d["k"]), d["cs"].double().cpu().numpy(), d["pos"].cpu().numpy(), False, "f16")
    assert torch.equal(vc.view(-1, H, D)[slots.long()], d["v"])


def test_no_tokens(pa):
    d = inputs(1, 2, 2, 64, 16, 64, "f16", 1)
    n = pa.pa_launch_count()
    pa.pa_cache_append_rope(d["k"][:0], d["v"][:0], d["slots"][:0], d["kc"], d["vc"], d["pos"][:0], d["cs"], q=d["q"][:0], q_out=d["q"][:0])
    assert pa.pa_launch_count() == n
