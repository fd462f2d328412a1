"""The README's example of windows and the 8-bit cache runs as written (GPU)."""

import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_third_python_example_runs(pa):
    text = open(os.path.join(ROOT, "README.md")).read()
    x = {}
    exec(compile(re.findall(r"```python\n(.*?)```", text, re.S)[2], "README.md", "exec"), x)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == 0
    for name in ("prompt", "one", "one8", "all8"):
        assert torch.isfinite(x[name]).all(), name
    # with a scale of 0 every token weighs the same: the mean of the values, each within half a step of the 8 bits
    mean = torch.cat([x["v"], x["v1"]]).float().mean(0).repeat_interleave(4, 0)
    even = pa.pa_decode_q8(x["q1"], x["k8"], x["v8"], x["k_step"], x["v_step"], x["tables"], x["lens"], 0.0, torch.empty_like(x["q1"]))
    used = x["tables"][0, : -(-9001 // 16)].long()
    assert (even[0].float() - mean).abs().max() <= 0.5 * x["v_step"][used].max() + 2.0 ** -8 * mean.abs().max()
    # a window over 9001 tokens sees what no window sees: one kernel's sums against the other's, of weights with 22 bits
    wide = pa.pa_decode_q8(x["q1"], x["k8"], x["v8"], x["k_step"], x["v_step"], x["tables"], x["lens"], 128 ** -0.5, torch.empty_like(x["q1"]), window=9001)
    assert (wide.float() - x["all8"].float()).abs().max() <= 2.0 ** -7 * x["all8"].float().abs().max()
