"""The cases of test_gpu_window_precision.py tell right from wrong: a mistake planted in the plain form leaves their tolerance (CPU)."""

import numpy as np
import pytest

from tests._window_precision_cases import carried, parts16, rounded, sink_and_steps, uneven_weights8, within

STEPS = [1.0, 1.0 + 2.0 ** -7, 2.0 - 2.0 ** -6, 0.0078125, 1 / 254]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("step", STEPS)
def test_weights_without_their_second_part_are_seen(dtype, D, step):
    q, k, v = uneven_weights8(1, D, step, D)
    assert within(rounded(carried(k, v, q), dtype), q[None], k, v, dtype).all()
    assert not within(carried(k, v, q, parts=1), q[None], k, v, dtype).any()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("step,others", [(1.0, 1.0), (1.0 + 2.0 ** -7, 1.0), (2.0 - 2.0 ** -6, 1.0), (4.0, 1.0), (4096.0, 2048.0)])
def test_small_weights_in_few_bits_are_seen(dtype, step, others):
    q, k, v = sink_and_steps(1, 64, 1000, step, others)
    assert within(rounded(carried(k, v, q), dtype), q[None], k, v, dtype).all()
    assert not within(carried(k, v, q, room=0), q[None], k, v, dtype).any()
    if step > 1000:                                # (the sink's own weight passes fp16's range)
        with np.errstate(over="ignore", invalid="ignore"):
            assert not within(carried(k, v, q, in_units=False), q[None], k, v, dtype).any()


def test_what_the_parts_leave_over_reaches_its_bound():
    """Where the largest step is a power of two, a weight that is held 2^7 higher is held 2^6 higher with it: it loses up to 2^-31 of
    the largest weight, and more than 2^-32."""
    w = np.exp(-np.linspace(15.0, 20.0, 400))
    worst = np.abs(parts16(w * 2.0 ** 6) / 2.0 ** 6 - w).max()
    assert 2.0 ** -32 < worst <= 2.0 ** -31
