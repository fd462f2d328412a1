"""Decode over the 4-bit cache and over selected frames where one rounding decides: each case's scores are exact in fp32
(GPU).  test_decode_precision_host.py shows that the tolerances see the mistakes they are for."""

import numpy as np
import pytest
import torch

from oracle.operators import attend, quantise_q4, values_q4
from tests._operators_common import TD, attention_tolerance, host64
from tests._precision_cases import fine_tolerance, one_sink, outlying_query, paged_rows, single_products, uneven_weights

pytestmark = pytest.mark.gpu


def decode_q4(pa, q, k4, v4, scale, dtype, B=16):
    """pa_decode_q4 of q [Hq, D] over rows [N, H, W] of one sequence -> [Hq, D] in 64 bits."""
    (kc, t), (vc, _) = (paged_rows(torch.from_numpy(x), B, 1) for x in (k4, v4))
    kc, vc = (c.transpose(1, 2).contiguous().cuda() for c in (kc, vc))
    qd = torch.from_numpy(q).to(TD[dtype])[None].cuda()
    assert np.array_equal(host64(qd[0]), q)
    out = torch.full_like(qd, float("nan"))
    lens = torch.tensor([len(k4)], dtype=torch.int32).cuda()
    pa.pa_decode_q4(qd, kc, vc, t.cuda(), lens, scale, out)
    assert pa.pa_get_device_status() == 0
    return host64(out[0])


def decode_selected(pa, q, k, v, scale, dtype, B=16):
    """pa_decode_selected of q [Hq, D] over all frames of one sequence's rows [N, H, D] -> [Hq, D] in 64 bits."""
    (kc, t), (vc, _) = (paged_rows(torch.from_numpy(x).to(TD[dtype]), B, 1) for x in (k, v))
    qd = torch.from_numpy(q).to(TD[dtype])[None].cuda()
    assert np.array_equal(host64(qd[0]), q)
    out = torch.full_like(qd, float("nan"))
    lens = torch.tensor([len(k)], dtype=torch.int32).cuda()
    sel = torch.arange(t.shape[1], dtype=torch.int32).repeat(1, k.shape[1], 1).cuda()
    pa.pa_decode_selected(qd, kc.cuda(), vc.cuda(), t.cuda(), lens, sel, scale, out)
    assert pa.pa_get_device_status() == 0
    return host64(out[0])


def decode(pa, call, q, k, v, scale, dtype):
    """Either call over the same numbers [N, H, D], which 4 bits hold as they are."""
    if call == "selected":
        return decode_selected(pa, q, k, v, scale, dtype)
    k4, v4 = (quantise_q4(x.astype(np.float32)) for x in (k, v))
    assert np.array_equal(values_q4(k4), k) and np.array_equal(values_q4(v4), v)
    return decode_q4(pa, q, k4, v4, scale, dtype)


def close(got, q, k, v, scale, dtype, weight_step, weight_tiny=0.0):
    err, tol = np.abs(got - attend(q, k, v, scale)), fine_tolerance(q, k, v, scale, dtype, weight_step, weight_tiny)
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))


# ---- the 4-bit cache's numbers ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 4, 8, 16])
def test_keys_are_the_numbers_that_codes_stand_for(pa, dtype, D, g):
    q, k4, v4 = single_products(2, g, D, 300, D + g)
    close(decode_q4(pa, q, k4, v4, 1.0, dtype), q, values_q4(k4), values_q4(v4), 1.0, dtype, 2.0 ** -22, 2.0 ** -32)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 4, 8, 16])
def test_small_queries_beside_an_outlying_one(pa, D, g):
    q, k4, v4 = outlying_query(2, g, D, 300, 1)
    close(decode_q4(pa, q, k4, v4, 1.0, "bf16"), q, values_q4(k4), values_q4(v4), 1.0, "bf16", 2.0 ** -22, 2.0 ** -32)


# ---- the weights -------------------------------------------------------------------------------------------
@pytest.mark.parametrize("call", ["q4", "selected"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 4, 8, 16])
def test_weights_keep_their_second_part(pa, call, dtype, D, g):
    part = "f16" if call == "q4" else dtype
    k, v = uneven_weights(2, D, TD[part], D + g)
    q = np.zeros((2 * g, D))
    q[:, [0, 32]] = 1.0
    close(decode(pa, call, q, k, v, 1.0, dtype), q, k, v, 1.0, dtype, 2.0 ** (-22 if part == "f16" else -16))


@pytest.mark.parametrize("call", ["q4", "selected"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("N", [60, 5000])
@pytest.mark.parametrize("g", [1, 8])
def test_small_weights_beside_a_sink(pa, call, dtype, N, g):
    k, v = one_sink(2, 64, N)
    q = np.zeros((2 * g, 64))
    q[:, 0] = 1.0
    bf16 = call == "selected" and dtype == "bf16"     # no least number to speak of
    close(decode(pa, call, q, k, v, 1.0, dtype), q, k, v, 1.0, dtype, 2.0 ** (-16 if bf16 else -22), 0.0 if bf16 else 2.0 ** -32)


# ---- infinities ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("g", [1, 4, 8, 16])
def test_scores_of_minus_infinity_weigh_nothing(pa, dtype, g):
    """The keys of a sequence's first tokens score -inf, over more than a tile; then all of them do."""
    for first, N in ((1, 20), (20, 40), (40, 3000), (0, 20)):
        gen = torch.Generator().manual_seed(first + g)
        k, v = (torch.randn(N, 2, 64, generator=gen).to(TD[dtype]).double().numpy() for _ in range(2))
        q = torch.randn(2 * g, 64, generator=gen).to(TD[dtype]).double().numpy()
        q[:, 3] = 1.0
        k[:first, :, 3] = -np.inf
        with np.errstate(invalid="ignore"):
            ref = attend(q, k, v, 0.125)
        rest = attend(q, k[first:], v[first:], 0.125)
        assert np.allclose(ref, rest, rtol=1e-12, atol=0)
        tol = attention_tolerance(rest, TD[dtype], q, k[first:], v[first:], 0.125, 2.0 ** (-22 if dtype == "f16" else -16))
        err = np.abs(decode_selected(pa, q, k, v, 0.125, dtype) - rest)
        assert (err <= tol).all(), (first, N, float(err.max()))
    k[:, :, 3] = -np.inf
    assert not decode_selected(pa, q, k, v, 0.125, dtype).any()   # as pa_decode leaves it


# ---- the range of the queries ------------------------------------------------------------------------------
@pytest.mark.parametrize("power", [120, 110, 99, 16, -100, -112, -120, -126])
@pytest.mark.parametrize("g", [1, 8])
def test_queries_over_the_whole_range_of_bf16(pa, power, g):
    """The same softmax whatever power of two the queries carry and the scale takes back: the same bits."""
    gen = torch.Generator().manual_seed(g)
    k4, v4 = (quantise_q4(torch.randn(200, 2, 64, generator=gen).numpy()) for _ in range(2))
    q = torch.rand(2 * g, 64, generator=gen).add(1.0).bfloat16().double().numpy() * np.where(np.arange(64) % 2, -1.0, 1.0)
    plain = decode_q4(pa, q, k4, v4, 2.0 ** -3, "bf16")
    assert np.array_equal(decode_q4(pa, q * 2.0 ** power, k4, v4, 2.0 ** (-3 - power), "bf16"), plain)
    ref = attend(q, values_q4(k4), values_q4(v4), 2.0 ** -3)
    assert (np.abs(plain - ref) <= attention_tolerance(ref, torch.bfloat16, q, values_q4(k4), values_q4(v4), 2.0 ** -3, 2.0 ** -22)).all()
