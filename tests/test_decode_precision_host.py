"""The cases of test_gpu_decode_precision.py tell right from wrong: a mistake planted in the plain form leaves their
tolerance (CPU)."""

import numpy as np
import pytest
import torch

from oracle.operators import attend, values_q4
from tests._operators_common import TD
from tests._precision_cases import fine_tolerance, one_sink, outlying_query, single_products, uneven_weights


def rounded(x, dtype):
    return torch.from_numpy(x).to(TD[dtype]).double().numpy()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 4, 8, 16])
def test_keys_that_are_not_rounded_are_seen(D, g):
    q, k4, v4 = single_products(2, g, D, 300, D + g)
    k, v = values_q4(k4), values_q4(v4)
    tol = fine_tolerance(q, k, v, 1.0, "bf16", 2.0 ** -11)
    assert (np.abs(rounded(attend(q, k, v, 1.0), "bf16") - attend(q, k, v, 1.0)) <= tol).all()
    wrong = attend(q, values_q4(k4, rounded=False), v, 1.0)
    assert (np.abs(wrong - attend(q, k, v, 1.0)) > tol).any()


def test_offsets_behind_an_outlying_query_are_seen():
    q, k4, v4 = outlying_query(2, 4, 128, 300, 1)
    k, v = values_q4(k4), values_q4(v4)
    s = k[:, 0] @ q[0]
    assert np.abs(s).max() > 8                     # the small elements decide the softmax
    tol = fine_tolerance(q, k, v, 1.0, "bf16", 2.0 ** -11)
    wrong = attend(np.where(q > 1, q, 0), k, v, 1.0)
    assert (np.abs(wrong - attend(q, k, v, 1.0)) > tol).any()


@pytest.mark.parametrize("part,dtype,step", [("f16", "f16", 2.0 ** -22), ("f16", "bf16", 2.0 ** -22), ("bf16", "bf16", 2.0 ** -16)])
@pytest.mark.parametrize("D", [64, 128])
def test_weights_without_their_second_part_are_seen(part, dtype, step, D):
    k, v = uneven_weights(1, D, TD[part], D)
    q = np.zeros((1, D))
    q[0, [0, 32]] = 1.0
    ref, tol = attend(q, k, v, 1.0), fine_tolerance(q, k, v, 1.0, dtype, step)
    w = np.exp(k[:, 0] @ q[0])
    wrong = rounded(w, part) @ v[:, 0] / w.sum()
    assert (np.abs(wrong - ref[0]) > 2 * tol[0]).all()
    both = (rounded(w, part) + rounded(w - rounded(w, part), part)) @ v[:, 0] / w.sum()
    assert (np.abs(rounded(both, dtype) - ref[0]) <= tol[0]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_small_weights_in_few_bits_are_seen(dtype):
    k, v = one_sink(1, 64, 1000)
    q = np.zeros((1, 64))
    q[0, 0] = 1.0
    ref, tol = attend(q, k, v, 1.0), fine_tolerance(q, k, v, 1.0, dtype, 2.0 ** -22, 2.0 ** -32)
    w = np.exp(k[:, 0] @ q[0])
    both = rounded(w, "f16") + rounded(w - rounded(w, "f16"), "f16")
    assert (np.abs(both @ v[:, 0] / w.sum() - ref[0]) > 10 * tol[0]).all()
