"""Refusals of the block-sparse calls beside those of test_operators_host.py (CPU)."""

import pytest
import torch

from test_operators_host import CUDA, F16, I32, STRIDE, Call, desc


@pytest.fixture()
def select(pa):
    if torch.cuda.is_available():
        pytest.skip("descriptors point at no memory: only where a call cannot launch")
    return Call(pa, "pa_select_blocks", q=desc(pa, F16, 2, 8, 64), b=desc(pa, F16, 4, 2, 2, 64), bt=desc(pa, I32, 2, 3), cl=desc(pa, I32, 2),
                B=16, first=1, last=1, sel=desc(pa, I32, 2, 2, 5), stream=None)


def test_lists_that_overlap_are_refused(pa, select):
    """Heads 8 apart and sequences 10: the second sequence's first list begins inside the first one's second."""
    assert select(sel=desc(pa, I32, 2, 2, 5, stride=(10, 8, 1))) == STRIDE
    assert select(sel=desc(pa, I32, 2, 2, 5, stride=(13, 8, 1))) == CUDA
    assert select(sel=desc(pa, I32, 1, 2, 5, stride=(10, 8, 1)), q=desc(pa, F16, 1, 8, 64), bt=desc(pa, I32, 1, 3), cl=desc(pa, I32, 1)) == CUDA
