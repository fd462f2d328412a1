"""Window decode and decode over the 8-bit cache where one rounding decides: scores are exact in fp32, or products of two such
numbers (GPU).  test_window_precision_host.py shows that the tolerances see the mistakes they are for."""

import numpy as np
import pytest
import torch

from oracle.operators import attend
from tests._operators_common import TD, attention_tolerance, host64
from tests._precision_cases import fine_tolerance, one_sink, paged_rows, uneven_weights
from tests._window_precision_cases import Rows8, hidden_between, sink_and_steps, tolerance8, uneven_weights8

pytestmark = pytest.mark.gpu


def queries(q, dtype):
    qd = torch.from_numpy(q).to(TD[dtype])[None].cuda()
    assert np.array_equal(host64(qd[0]), q)
    return qd


def decode_window(pa, q, k, v, scale, dtype, sinks=0, gap=0, B=16):
    """pa_decode_window of q [Hq, D] over one sequence's rows [N, H, D], all of them seen: the first `sinks` through the
    sinks, the others through the window, `gap` rows between that are not."""
    rows = [hidden_between(x, sinks, gap, 7.0) for x in (k, v)]
    (kc, t), (vc, _) = (paged_rows(torch.from_numpy(x).to(TD[dtype]), B, 1) for x in rows)
    qd = queries(q, dtype)
    out = torch.full_like(qd, float("nan"))
    lens = torch.tensor([len(rows[0])], dtype=torch.int32).cuda()
    pa.pa_decode_window(qd, kc.cuda(), vc.cuda(), t.cuda(), lens, len(k) - sinks, scale, out, sinks=sinks)
    assert pa.pa_get_device_status() == 0
    return host64(out[0])


def decode_q8(pa, q, k, v, scale, dtype, window=0, B=16):
    """pa_decode_q8 of q [Hq, D] over rows of the 8-bit cache (Rows8), the last `window` of them."""
    caches = []
    for x in (k, v):
        cache, t = paged_rows(torch.from_numpy((x.codes + 128).astype(np.uint8)), B, 1)
        steps = torch.full((cache.shape[0], x.codes.shape[1]), float("nan"))
        steps[t[0].long()] = torch.from_numpy(x.steps[::B])
        caches += [cache.transpose(1, 2).contiguous().cuda(), steps.cuda()]
    qd = queries(q, dtype)
    out = torch.full_like(qd, float("nan"))
    lens = torch.tensor([len(k.codes)], dtype=torch.int32).cuda()
    pa.pa_decode_q8(qd, caches[0], caches[2], caches[1], caches[3], t.cuda(), lens, scale, out, window=window)
    assert pa.pa_get_device_status() == 0
    return host64(out[0])


def close(got, ref, tol):
    err = np.abs(got - ref)
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))


def close8(got, q, k, v, scale, dtype):
    close(got, attend(q, k.values(), v.values(), scale), tolerance8(q, k, v, scale, dtype))


# ---- windows ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,step", [("f16", 2.0 ** -22), ("bf16", 2.0 ** -16)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 4, 8, 16])
@pytest.mark.parametrize("sinks,gap", [(0, 21), (19, 40)])
def test_window_weights_keep_their_second_part(pa, dtype, step, D, g, sinks, gap):
    k, v = uneven_weights(2, D, TD[dtype], D + g)
    q = np.zeros((2 * g, D))
    q[:, [0, 32]] = 1.0
    got = decode_window(pa, q, k, v, 1.0, dtype, sinks, gap)
    close(got, attend(q, k, v, 1.0), fine_tolerance(q, k, v, 1.0, dtype, step))


@pytest.mark.parametrize("dtype,step,least", [("f16", 2.0 ** -22, 2.0 ** -32), ("bf16", 2.0 ** -16, 0.0)])
@pytest.mark.parametrize("N", [60, 5000])
@pytest.mark.parametrize("g", [1, 8, 16])
def test_window_small_weights_beside_a_sink(pa, dtype, step, least, N, g):
    k, v = one_sink(2, 64, N)
    q = np.zeros((2 * g, 64))
    q[:, 0] = 1.0
    got = decode_window(pa, q, k, v, 1.0, dtype, 5, 100)
    close(got, attend(q, k, v, 1.0), fine_tolerance(q, k, v, 1.0, dtype, step, least))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("g", [1, 4, 8, 16])
def test_window_scores_of_minus_infinity_weigh_nothing(pa, dtype, g):
    for first, N in ((1, 20), (20, 40), (40, 3000), (0, 20)):
        gen = torch.Generator().manual_seed(first + g)
        k, v = (torch.randn(N, 2, 64, generator=gen).to(TD[dtype]).double().numpy() for _ in range(2))
        q = torch.randn(2 * g, 64, generator=gen).to(TD[dtype]).double().numpy()
        q[:, 3] = 1.0
        k[:first, :, 3] = -np.inf
        rest = attend(q, k[first:], v[first:], 0.125)
        tol = attention_tolerance(rest, TD[dtype], q, k[first:], v[first:], 0.125, 2.0 ** (-22 if dtype == "f16" else -16))
        close(decode_window(pa, q, k, v, 0.125, dtype, 3, 30), rest, tol)
    k[:, :, 3] = -np.inf
    assert not decode_window(pa, q, k, v, 0.125, dtype).any()


# ---- the 8-bit cache -------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 4, 8, 16])
@pytest.mark.parametrize("step", [1.0, 1.0 + 2.0 ** -7, 2.0 - 2.0 ** -6, 0.0078125, 1 / 254])
def test_8_bit_weights_keep_their_second_part(pa, dtype, D, g, step):
    one, k, v = uneven_weights8(2, D, step, D + g)
    q = np.tile(one, (2 * g, 1))
    close8(decode_q8(pa, q, k, v, 1.0, dtype), q, k, v, 1.0, dtype)
    more = [Rows8(hidden_between(x.codes, 0, 48, 99), hidden_between(x.steps, 0, 48, 3.0)) for x in (k, v)]
    close8(decode_q8(pa, q, *more, 1.0, dtype, window=64), q, k, v, 1.0, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("N", [64, 5000])
@pytest.mark.parametrize("g", [1, 8, 16])
@pytest.mark.parametrize("step,others", [(1.0, 1.0), (1.0 + 2.0 ** -7, 1.0), (2.0 - 2.0 ** -6, 1.0), (4.0, 1.0), (4096.0, 2048.0)])
def test_8_bit_small_weights_beside_a_sink(pa, dtype, N, g, step, others):
    one, k, v = sink_and_steps(2, 64, N, step, others)
    q = np.tile(one, (2 * g, 1))
    close8(decode_q8(pa, q, k, v, 1.0, dtype), q, k, v, 1.0, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 4, 8, 16])
def test_8_bit_scores_are_codes_times_steps(pa, dtype, D, g):
    """Queries of one element: a score is one product of query, code and step, up to about +-60; steps of each frame its own."""
    rng = np.random.default_rng(D + g)
    N, H = 320, 2
    codes = rng.integers(100, 128, (N, H, D)) * rng.choice([-1, 1], (1, 1, D))
    k = Rows8(codes, np.repeat(1 / rng.integers(128, 256, (N // 16, H)).astype(np.float32) * np.float32(0.25), 16, 0) * np.float32(64))
    v = Rows8(rng.integers(-127, 128, (N, H, D)), np.repeat(1 / rng.integers(128, 256, (N // 16, H)).astype(np.float32), 16, 0))
    q = np.zeros((H * g, D))
    for j in range(len(q)):
        d = int(rng.integers(D))
        q[j, d] = float(torch.tensor(60.0 / np.abs(k.values()[:, :, d]).max()).bfloat16())
    close8(decode_q8(pa, q, k, v, 1.0, dtype), q, k, v, 1.0, dtype)


@pytest.mark.parametrize("power", [120, 110, 99, 16, -100, -112, -120, -126])
@pytest.mark.parametrize("g", [1, 8, 16])
def test_8_bit_queries_over_the_whole_range_of_bf16(pa, power, g):
    """The same softmax whatever power of two the queries carry and the scale takes back: the same bits."""
    gen = torch.Generator().manual_seed(g)
    k, v = (Rows8(torch.randint(-127, 128, (208, 2, 64), generator=gen).numpy(), np.full((208, 2), 1 / 140, np.float32)) for _ in range(2))
    q = torch.rand(2 * g, 64, generator=gen).add(1.0).bfloat16().double().numpy() * np.where(np.arange(64) % 2, -1.0, 1.0)
    plain = decode_q8(pa, q, k, v, 2.0 ** -3, "bf16")
    assert np.array_equal(decode_q8(pa, q * 2.0 ** power, k, v, 2.0 ** (-3 - power), "bf16"), plain)
    ref = attend(q, k.values(), v.values(), 2.0 ** -3)
    close(plain, ref, attention_tolerance(ref, torch.bfloat16, q, k.values(), v.values(), 2.0 ** -3, 2.0 ** -22))
